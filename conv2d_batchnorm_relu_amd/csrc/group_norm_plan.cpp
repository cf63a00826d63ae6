// group_norm_plan.cpp -- how a group norm call is laid out: groups, pixels and images a workgroup, and
// whether an image is held whole or in tiles.
#include <algorithm>

#include "block_launch.h"
#include "group_norm.h"

namespace cbr {
namespace gnorm {
namespace {

// Expected time of a layout in us, fitted to some 15000 measurements (450 calls of 235 shapes, both passes, 33 layouts each in the
// mean; the layout it picks takes 4% longer than the fastest one in the mean, 6% on 272 calls that were not in the fit, 2.4
// times as long at worst).  Workgroups run in rounds of as many as the registers let share the CUs; in a round a CU's loads
// and stores and its arithmetic overlap only in part, and a workgroup alone on its CU loads, sums and stores one after the other.
double expected_us(const cbr_group_norm_shape &s, const Geo &g, bool backward, int cpg, int nv, int size)
{
    auto up = [](double a, double b) { return (double)(int64_t)((a + b - 1) / b); };
    const int f = 4 / size, t = threads_of(g);
    const bool tiled = g.tiles > 1;
    const int waves = tiled ? (backward ? 20 : 32) : backward ? (g.k <= f ? 24 : g.k <= 2 * f ? 20 : 16) : g.k <= 2 * f ? 32 : g.k <= 4 * f ? 24 : 16;
    const double share = std::max(1, waves * 64 / std::max(t, 64)), wgs = (double)workgroups(s, g);
    const double act = std::min(share, up(wgs, 256.)), waves_of = up(t, 64.);
    const double values = (double)g.ipw * std::min<int64_t>(s.pixels, (int64_t)g.P * g.k) * g.ng * cpg;
    // memory: bytes over what a CU gets, 30 or 37 GB/s or its share of 5 TB/s, and what its loads in flight carry
    const double width = (double)g.ng * cpg * size;
    const double narrow = width >= 128 ? 1. : width >= 64 ? 1.02 : width >= 32 ? 1.28 : 1.55;   // runs of a part of a line
    const double passes = tiled ? (backward ? 5. : 3.) : backward ? 3. : 2.;
    const double flying = t * act * (tiled ? std::min<double>(g.k, 1.5) / 0.6 : g.k / 0.165) * (backward ? 2. : 1.) * 8 * size;
    const double rate = std::min(std::min(tiled ? 29.5e3 : 37e3, flying), 5.0e6 / std::min(wgs, 256.));
    const double mem = act * values * size * passes * narrow / rate;
    // arithmetic: instructions a value and pass
    const double ins = (s.act == CBR_ACT_SILU ? (backward ? 41. : 21.4) : backward ? 13. : 9.) * (nv > 1 ? 5. : 1.);
    const double alu = std::max(1., waves_of * act / 4.) * g.k * ins * (tiled ? 0.00073 : 0.0026);
    // the sums over a workgroup, and what the second kernel of large images reads before it begins
    const double sums = 0.113 * (tiled ? 2 : 1) * (g.pre ? 1 : 2) * up(t, 256.);
    const double join = !tiled ? 0. : 0.28 * up(g.tiles, 64.) * (backward ? up(g.V * 128., t) : up(g.ng, std::max(t / 64, 1)));
    const double rounds = std::max(1., wgs / (256. * share)), whole = rounds < 6. ? 0.08 * up(wgs, 256. * share) + 0.92 * rounds : rounds;
    double one = 0.52 + sums + join + std::max(mem, alu) + (tiled ? 0.09 : 2.25) * std::min(mem, alu);
    if (!tiled && act == 1. && rounds > 1.) one += 0.09 * mem;
    // (large maps by fewer than eight waves a CU: 4 x 112 x 112 x 512 backward 70 us, with eight 52)
    if (tiled && t * act < 512 && (double)s.images * s.pixels * s.channels * size > 32e6) one *= 1.1;
    return 4.7 + (tiled ? 1.4 : 0.) + (backward && s.images * g.tiles > 1 ? (tiled ? 0.8 : 3.9) : 0.) + whole * one;
}

Geo least_time(const cbr_group_norm_shape &s, bool backward)
{
    const int cpg = s.channels / s.groups, size = s.type == CBR_F32 ? 4 : 2, nv = split_of(cpg);
    const int most = (backward ? bwd_most(nv) : fwd_most(nv)) * 4 / size;   // pixels a thread holds of images held whole
    const int64_t limit = 0x7fffffff / ((int64_t)s.channels * size);        // pixels within 2^31 bytes
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    Geo best{};
    double least = 0;
    // Chunks of 1, 2, 4, ... groups, and of all (a call plans anew: few candidates).  Every chunk has eight
    // channels at least, if there are that many: else one of some groups more.  Runs of more than 1 KB only where there is
    // nothing else: of 203 calls measured both ways 24 were faster in them, 0.6% in the mean (most: 3 x 5735 x 1056 f32, 54 -> 44).
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
        const bool pow2 = (V & (V - 1)) == 0;
        for (int threads = 64; threads <= 1024; threads *= 2) {
            if (threads < V && threads < 1024) continue;
            Geo g{};
            g.V = V;
            g.ng = ng;
            g.chunks = chunks;
            g.P = std::max(1, threads / V);
            while (g.P > 1 && (g.P / 2 >= s.pixels || g.P > limit)) g.P = pow2 ? g.P / 2 : (g.P + 1) / 2;
            g.pre = pow2 && V <= 64 && V * g.P % 64 == 0;
            auto weigh = [&]() {
                if ((backward ? bwd_floats(g, cpg) : sum_floats(g, nv, 1)) > 40 * 1024) return;   // floats: a CU's 160 KB
                const double time = expected_us(s, g, backward, cpg, nv, size);
                if (least == 0 || time < least) {
                    least = time;
                    best = g;
                }
            };
            // Offsets of pixels past a part's end are formed too (their loads are switched off): of images held whole up to the
            // last turn's end, of tiles two turns more (see the kernels' loops).
            const int64_t k = up(s.pixels, g.P), held = k * g.P;
            g.ipw = (int)std::max<int64_t>(1, std::min<int64_t>({threads / (V * g.P), s.images, (limit - held) / s.pixels + 1}));
            if (k <= most && (g.ipw - 1) * s.pixels + held <= limit) {
                g.tiles = 1;
                g.k = (int)k;
                weigh();
            }
            // tiles for one, two or four workgroups a CU (a small call is not worth a second kernel, nor weighing it)
            g.ipw = 1;
            const int64_t turns = limit / g.P - 2;   // of a tile, at most
            if (turns < 1 || V * g.P < 64 || threads < 256 || k < 2 || (least > 0 && (double)s.images * s.pixels * s.channels < 250e3)) continue;
            for (int64_t total = 256; total <= 1024; total *= 2) {
                const int64_t tiles = std::max<int64_t>({2, up(s.pixels, g.P * turns), std::min<int64_t>(k, total / (s.images * chunks))});
                g.k = (int)up(s.pixels, tiles * g.P);
                g.tiles = (int)up(s.pixels, (int64_t)g.P * g.k);
                if (g.tiles > 1) weigh();
            }
        }
        if (ng == s.groups) break;
    }
    return best;
}

}  // namespace

// Weighing the layouts takes 1.5 us, half of what a launch does, and a layer asks with the same sizes again and again:
// each thread remembers the layouts of the last sizes.
Geo plan_group_norm(const cbr_group_norm_shape &s, bool backward)
{
    struct Known {
        int64_t images, pixels;
        int channels, groups, type, act, backward;
        Geo g;
    };
    static thread_local Known known[64];   // (zeros: no call has 0 images)
    uint64_t h = (uint64_t)s.images * 0x9E3779B97F4A7C15u + (uint64_t)s.pixels;
    h = (h * 0x9E3779B97F4A7C15u + (uint32_t)s.channels) * 0x9E3779B97F4A7C15u + (uint32_t)(s.groups * 32 + s.type * 8 + s.act * 2 + backward);
    Known &k = known[h * 0x9E3779B97F4A7C15u >> 58];
    if (k.images != s.images || k.pixels != s.pixels || k.channels != s.channels || k.groups != s.groups || k.type != s.type ||
        k.act != s.act || k.backward != (int)backward)
        k = Known{s.images, s.pixels, s.channels, s.groups, s.type, s.act, backward, least_time(s, backward)};
    return k.g;
}

}  // namespace gnorm
}  // namespace cbr
