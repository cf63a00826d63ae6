// group_norm_fwd.hip -- group norm with an activation over channels-last maps:
//   y = act((x - mean) / sqrt(var + eps) * w + b),  mean and var of an image's group of channels
// A workgroup holds whole groups of an image in registers from the load to the store, so x is read
// once, and the squared deviations are summed after the mean (no difference of large sums).  Where an
// image is too large for that, one kernel leaves every tile's (mean, M2), joined exactly by the
// formula of Chan, Golub and LeVeque, and a second one reads x again.
#include "block_launch.h"
#include "group_norm.h"

namespace cbr {
namespace {

using namespace gnorm;

template <int NV>
struct Coef {
    float mean[NV], a[8], b[8];   // u = (x - mean) a + b; SiLU: -log2(e) times that
    // a, b: w and b as they were given
    __device__ __forceinline__ void set(const float (&inv)[NV], const Split<NV> &sp, int act)
    {
        const float c = act == CBR_ACT_SILU ? -LOG2E : 1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            a[e] *= sp.pick(inv, e) * c;
            b[e] *= c;
        }
    }
    __device__ __forceinline__ void apply(float (&v)[8], const Split<NV> &sp, int act) const
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(v[e] - sp.pick(mean, e), a[e], b[e]);
        if (act == CBR_ACT_RELU) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = v[e] < 0.f ? 0.f : v[e];   // a NaN stays one
        } else if (act == CBR_ACT_SILU) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
            float power;
            v[e] *= scaled_sigmoid(v[e], power);
        }
        }
    }
};

// The thread of a group's first channel and pixel leaves its two values at out[group * stride].
template <int NV>
__device__ __forceinline__ void leave_groups(const GroupNormArgs &p, const Place &at, const Thread &me, const Split<NV> &sp, float *out,
                                             int64_t stride, const float (&u)[NV], const float (&v)[NV])
{
    if (me.prow == 0 && me.on)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = 8 * me.vec + e;
            if (c < at.w && c % p.cpg == 0) *(f32x2 *)(out + c / p.cpg * stride) = f32x2{sp.pick(u, e), sp.pick(v, e)};
        }
}

// Images held whole.  Bound by memory (256 x 28 x 28 x 512 bf16: 84 us, 4.9 TB/s; a large copy reaches 5.0), small calls by
// a chain of latencies: the load, two sums over the workgroup, the store (49 x 512: 5.5 us).
template <typename T, Tail TAIL, int NV, int K>
__global__ __launch_bounds__(1024) void gn_fwd_kernel(GroupNormArgs p)
{
    extern __shared__ __attribute__((aligned(16))) float lds[];
    const Place at(p);
    const Geo &g = p.g;
    const Thread me(p, at);
    const int row = me.sub * (int)p.pixels + me.prow;
    const Part<T, TAIL> in(p.x, me.first, row, p.C, g.P, me.vec, at.w);
    Raw8<T> raw[K];
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (i < g.k) in.load(raw[i], i, i * g.P < me.left);
    GroupSum<NV, 1> sum(p, lds, me);
    const Split<NV> sp(me.vec, p.cpg, at.ngl);
    const float count = (float)p.pixels * (float)p.cpg;
    Coef<NV> cf;
    float c[8] = {}, s[1][NV];
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (i < g.k) {   // (what is not there was loaded as zeros)
            float v[8];
            in.settle(raw[i]);
            unpack8<T>(raw[i], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) c[e] += v[e];
        }
    sp.collapse(c, s[0]);
    sum(s, sp);
#pragma unroll
    for (int e = 0; e < NV; ++e) cf.mean[e] = s[0][e] / count;
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = 0.f;
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (i < g.k && i * g.P < me.left) {
            float v[8];
            unpack8<T>(raw[i], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = v[e] - sp.pick(cf.mean, e);
                c[e] = fmaf(d, d, c[e]);
            }
        }
    if (TAIL != WHOLE)
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = 8 * me.vec + e < at.w ? c[e] : 0.f;
    // (asked for beside the second sum)
    load_vec<8, TAIL>(p.w ? p.w + at.c0 : nullptr, 1.f, me.vec, g.V, at.w, cf.a);
    load_vec<8, TAIL>(p.b ? p.b + at.c0 : nullptr, 0.f, me.vec, g.V, at.w, cf.b);
    sp.collapse(c, s[0]);
    sum(s, sp);
#pragma unroll
    for (int e = 0; e < NV; ++e) s[0][e] = 1.f / sqrtf(s[0][e] / count + p.eps);
    if (p.stats) leave_groups<NV>(p, at, me, sp, p.stats + (me.image * p.G + at.chunk * g.ng) * 2, 2, cf.mean, s[0]);
    cf.set(s[0], sp, p.act);
    const Part<T, TAIL> out(p.out, me.first, row, p.C, g.P, me.vec, at.w);
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (i < g.k) {
            float v[8];
            unpack8<T>(raw[i], v);
            cf.apply(v, sp, p.act);
            out.store(v, i, i * g.P < me.left, p.nt);
        }
}

// First kernel of large images: each group's (mean, M2) of a tile.  A thread runs the mean and the squares about it of every
// channel over its pixels (Welford's recurrence: eight chains side by side).  One pixel is on its way while another is
// added: more of them cost waves (four and four, bf16: 4 x 112 x 112 x 480 48 us; one and one 34, both in the layout of that
// time; the one that expected_us picks now takes 42).
template <typename T, Tail TAIL, int NV>
__global__ __launch_bounds__(1024) void gn_fwd_tiles_kernel(GroupNormArgs p)
{
    extern __shared__ __attribute__((aligned(16))) float lds[];
    const Place at(p);
    const Geo &g = p.g;
    const Thread me(p, at);
    const Part<T, TAIL> in(p.x, me.first, me.prow, p.C, g.P, me.vec, at.w);
    const int own = me.pixels(g);
    float mean[8] = {}, m2[8] = {}, n = 0.f;
    Raw8<T> one, two;
    auto add = [&](Raw8<T> &raw, int i) __attribute__((always_inline)) {
        if (i >= own) return;
        float v[8];
        in.settle(raw);
        unpack8<T>(raw, v);
        n += 1.f;
        const float share = 1.f / n;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = v[e] - mean[e];
            mean[e] = fmaf(d, share, mean[e]);
            m2[e] = fmaf(d, v[e] - mean[e], m2[e]);
        }
    };
    in.load(one, 0, 0 < own);
    for (int i = 0; i < g.k; i += 2) {
        in.load(two, i + 1, i + 1 < own);
        add(one, i);
        in.load(one, i + 2, i + 2 < own);
        add(two, i + 1);
    }
    // Over the channels and threads: the mean of the means, then the squares about it
    GroupSum<NV, 1> sum(p, lds, me);
    const Split<NV> sp(me.vec, p.cpg, at.ngl);
    const float count = (float)min((int64_t)g.P * g.k, p.pixels - (int64_t)at.tile * g.P * g.k) * (float)p.cpg;
    float c[8], s[1][NV], all[NV];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = n > 0.f ? mean[e] * n : 0.f;   // (a thread without pixels: 0 times nothing)
    sp.collapse(c, s[0]);
    sum(s, sp);
#pragma unroll
    for (int e = 0; e < NV; ++e) all[e] = s[0][e] / count;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float d = mean[e] - sp.pick(all, e);
        c[e] = n > 0.f && 8 * me.vec + e < at.w ? fmaf(d * d, n, m2[e]) : 0.f;
    }
    sp.collapse(c, s[0]);
    sum(s, sp);
    leave_groups<NV>(p, at, me, sp, p.part + ((me.image * p.G + at.chunk * g.ng) * g.tiles + at.tile) * 2, 2 * g.tiles, all, s[0]);
}

// Second kernel of large images: the tiles' statistics joined, then the tile's y.  (16 x 225 x 1001 f32 in 7 groups: 9.0 us
// for the first kernel and 9.2 for this one, of which reading and writing takes 2.9 and 5.7: rows of 143 channels leave four
// small workgroups a CU, all in the same phase.)
template <typename T, Tail TAIL, int NV>
__global__ __launch_bounds__(1024) void gn_fwd_apply_kernel(GroupNormArgs p)
{
    extern __shared__ __attribute__((aligned(16))) float lds[];   // [ng][2]
    const Place at(p);
    const Geo &g = p.g;
    const Thread me(p, at);
    const Part<T, TAIL> in(p.x, me.first, me.prow, p.C, g.P, me.vec, at.w), out(p.out, me.first, me.prow, p.C, g.P, me.vec, at.w);
    const int own = me.pixels(g);
    Raw8<T> one, two;
    in.load(one, 0, 0 < own);
    Coef<NV> cf;
    load_vec<8, TAIL>(p.w ? p.w + at.c0 : nullptr, 1.f, me.vec, g.V, at.w, cf.a);
    load_vec<8, TAIL>(p.b ? p.b + at.c0 : nullptr, 0.f, me.vec, g.V, at.w, cf.b);
    // A wave a group, its lanes the tiles (asked for once, where 64 hold them): the mean by its distance from the
    // first tile's, then M2
    const int t = threadIdx.x, lane = t & 63, waves = blockDim.x >> 6;   // (whole ones, at least one)
    const int64_t per_tile = (int64_t)g.P * g.k;
    const float all = (float)p.pixels, each = (float)per_tile, last = (float)(p.pixels - (g.tiles - 1) * per_tile);
    if (t >> 6 < waves)
        for (int j = t >> 6; j < at.ngl; j += waves) {
            const f32x2 *part = (const f32x2 *)p.part + (me.image * p.G + at.chunk * g.ng + j) * g.tiles;
            const f32x2 own = part[min(lane, g.tiles - 1)];
            const float m0 = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(own[0])));
            float d = 0.f, m2 = 0.f;
            for (int i = lane; i < g.tiles; i += 64)
                d = fmaf((i + 1 < g.tiles ? each : last) / all, (i == lane ? own[0] : part[i][0]) - m0, d);
            const float mean = m0 + wave_sum(d);
            for (int i = lane; i < g.tiles; i += 64) {
                const f32x2 q = i == lane ? own : part[i];
                const float e = q[0] - mean;
                m2 += q[1] + e * e * ((i + 1 < g.tiles ? each : last) * (float)p.cpg);
            }
            const float inv = 1.f / sqrtf(wave_sum(m2) / (all * (float)p.cpg) + p.eps);
            if (lane == 0) {
                lds[2 * j] = mean;
                lds[2 * j + 1] = inv;
                if (at.tile == 0 && p.stats) *(f32x2 *)(p.stats + (me.image * p.G + at.chunk * g.ng + j) * 2) = f32x2{mean, inv};
            }
        }
    const Split<NV> sp(me.vec, p.cpg, at.ngl);
    __syncthreads();
    float inv[NV];
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        cf.mean[e] = lds[2 * sp.gi[e]];
        inv[e] = lds[2 * sp.gi[e] + 1];
    }
    cf.set(inv, sp, p.act);
    auto finish = [&](Raw8<T> &raw, int i) __attribute__((always_inline)) {
        float v[8];
        in.settle(raw);
        unpack8<T>(raw, v);
        cf.apply(v, sp, p.act);
        out.store(v, i, i < own, p.nt);
    };
    for (int i = 0; i < g.k; i += 2) {
        in.load(two, i + 1, i + 1 < own);
        finish(one, i);
        in.load(one, i + 2, i + 2 < own);
        finish(two, i + 1);
    }
}

template <typename Kern>
hipError_t launch_with(Kern k, const GroupNormArgs &a, int lds, hipStream_t st)
{
    const Geo &g = a.g;
    const uint32_t grid = (uint32_t)((a.images + g.ipw - 1) / g.ipw * g.tiles * g.chunks);
    const hipError_t e = raise_lds_limit((const void *)k, lds);
    if (e != hipSuccess) return e;
    return launch(k, dim3(grid), dim3(threads_of(g)), lds, st, nullptr, nullptr, a);
}

template <typename T, Tail TAIL, int NV>
hipError_t launch_tail(const GroupNormArgs &a, hipStream_t st)
{
    constexpr int B = 4 / T::SIZE;   // a vector takes 4 registers of 16-bit types, 8 of fp32
    const int lds = sum_floats(a.g, NV, 1) * (int)sizeof(float), k = a.g.k;
    if (a.g.tiles > 1) {
        const hipError_t e = launch_with(gn_fwd_tiles_kernel<T, TAIL, NV>, a, lds, st);
        if (e != hipSuccess) return e;
        return launch_with(gn_fwd_apply_kernel<T, TAIL, NV>, a, 2 * a.g.ng * (int)sizeof(float), st);
    }
    if (k <= 2 * B) return launch_with(gn_fwd_kernel<T, TAIL, NV, 2 * B>, a, lds, st);
    if (k <= 4 * B) return launch_with(gn_fwd_kernel<T, TAIL, NV, 4 * B>, a, lds, st);
    if (NV < 8 && k <= 7 * B) return launch_with(gn_fwd_kernel<T, TAIL, NV, 7 * B>, a, lds, st);
    return launch_with(gn_fwd_kernel<T, TAIL, NV, fwd_most(NV) * B>, a, lds, st);
}

template <typename T>
hipError_t launch_type(const GroupNormArgs &a, hipStream_t st)
{
    if (a.cpg % 8 == 0) return launch_tail<T, WHOLE, 1>(a, st);
    const bool whole = a.C % 8 == 0 && (a.g.chunks == 1 || a.g.ng * a.cpg % 8 == 0);
    if (a.cpg > 8) return whole ? launch_tail<T, WHOLE, 2>(a, st) : launch_tail<T, PART, 2>(a, st);
    if (whole) return launch_tail<T, WHOLE, 8>(a, st);
    return a.C >= 8 ? launch_tail<T, PART, 8>(a, st) : launch_tail<T, SHORT, 8>(a, st);   // (shorter: one chunk)
}

}  // namespace

hipError_t launch_group_norm_fwd(const cbr_group_norm_shape &s, const GroupNormArgs &a, hipStream_t st)
{
    if (s.type == CBR_BF16) return launch_type<Bf16>(a, st);
    if (s.type == CBR_F16) return launch_type<F16>(a, st);
    return launch_type<F32>(a, st);
}

}  // namespace cbr
