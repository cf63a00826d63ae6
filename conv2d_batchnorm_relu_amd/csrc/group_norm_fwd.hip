// group_norm_fwd.hip -- group norm with an activation over channels-last maps:
//   y = act((x - mean) / sqrt(var + eps) * w + b),  mean and var of an image's group of channels
// A workgroup holds whole groups of an image in registers from the load to the store, so x is read
// once, and the squared deviations are summed after the mean (no difference of large sums).  Where an
// image is too large for that, one kernel leaves every tile's (mean, M2), joined exactly by the
// formula of Chan, Golub and LeVeque, and a second one reads x again, last tile first.
#include "block_launch.h"
#include "group_norm.h"

namespace cbr {
namespace {

using namespace gnorm;

template <Tail TAIL, int NV>
struct Coef {
    float mean[NV], a[8], b[8];   // y = act((x - mean) a + b)
    __device__ __forceinline__ void apply(float (&v)[8], int act) const
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(v[e] - mean[NV == 1 ? 0 : e], a[e], b[e]);
        if (act == CBR_ACT_RELU) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = v[e] < 0.f ? 0.f : v[e];   // a NaN stays one
        } else if (act == CBR_ACT_SILU) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= sigmoid(v[e]);
        }
    }
};

// TILES: leaves each group's (mean, M2) of this tile instead of y.
template <typename T, Tail TAIL, int NV, int K, bool TILES>
__global__ __launch_bounds__(1024) void gn_fwd_kernel(GroupNormArgs p)
{
    extern __shared__ __attribute__((aligned(16))) float lds[];
    const Place<false> at(p, gridDim.x);
    const Geo &g = p.g;
    const int t = threadIdx.x, vec = t % g.V, q = t / g.V, prow = q % g.P, sub = q / g.P;
    const int64_t image = at.image + sub, first = (int64_t)at.tile * g.P * g.k;
    const int64_t rows = min((int64_t)g.P * g.k, p.pixels - first);   // of this tile
    const bool on = image < p.images;
    const int left = (int)(rows - prow);                               // pixels prow, prow + P, ... below it
    const int64_t start = ((image * p.pixels + first + prow) * p.C + at.c0) * T::SIZE, step = (int64_t)g.P * p.C * T::SIZE;
    Row<T, 8, TAIL> raw[K];
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (i < g.k) raw[i].load((const char *)p.x + start + i * step, vec, g.V, at.w, on && i * g.P < left);
    Coef<TAIL, NV> cf;
    if constexpr (!TILES) {
        load_vec<8, TAIL>(p.w ? p.w + at.c0 : nullptr, 1.f, vec, g.V, at.w, cf.a);
        load_vec<8, TAIL>(p.b ? p.b + at.c0 : nullptr, 0.f, vec, g.V, at.w, cf.b);
    }
    GroupSum<NV> sum(p, lds, vec, prow, sub);
    int gi[NV];
    groups_of<NV>(vec, p.cpg, at.ngl, gi);
    const float count = (float)rows * (float)p.cpg;

    float s[NV] = {};
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (i < g.k) {   // (what is not there was loaded as zeros)
            float v[8];
            raw[i].get(v, vec, g.V, at.w);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[NV == 1 ? 0 : e] += v[e];
        }
    sum(s, gi);
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        cf.mean[e] = s[e] / count;
        s[e] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (i < g.k) {
            float v[8], u[NV] = {};
            raw[i].get(v, vec, g.V, at.w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = v[e] - cf.mean[NV == 1 ? 0 : e];
                u[NV == 1 ? 0 : e] = fmaf(d, d, u[NV == 1 ? 0 : e]);
            }
#pragma unroll
            for (int e = 0; e < NV; ++e) s[e] += i * g.P < left ? u[e] : 0.f;
        }
    sum(s, gi);
    // (columns of vectors past the chunk are of no group)
    float *const mine = TILES ? p.part + ((image * g.tiles + at.tile) * p.G + at.chunk * g.ng) * 2
                              : p.stats ? p.stats + (image * p.G + at.chunk * g.ng) * 2 : nullptr;
    // One thread of each group's first channels has what its statistics are
    if (on && prow == 0 && mine && 8 * vec < at.w)
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            const int c = 8 * vec + e;
            if (c < at.w && c % p.cpg == 0)
                *(f32x2 *)(mine + 2 * gi[e]) = TILES ? f32x2{cf.mean[e], s[e]} : f32x2{cf.mean[e], 1.f / sqrtf(s[e] / count + p.eps)};
        }
    if constexpr (!TILES) {
#pragma unroll
        for (int e = 0; e < 8; ++e) cf.a[e] *= 1.f / sqrtf(s[NV == 1 ? 0 : e] / count + p.eps);
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (i < g.k) {
                float v[8];
                raw[i].get(v, vec, g.V, at.w);
                cf.apply(v, p.act);
                if (on && i * g.P < left) Row<T, 8, TAIL>::store((char *)p.out + start + i * step, vec, g.V, at.w, v);
            }
    }
}

// Second kernel of large images: the tiles' statistics joined, then the tile's y.
template <typename T, Tail TAIL, int NV, int K>
__global__ __launch_bounds__(1024) void gn_fwd_apply_kernel(GroupNormArgs p)
{
    extern __shared__ __attribute__((aligned(16))) float lds[];   // [ng][2]
    const Place<true> at(p, gridDim.x);
    const Geo &g = p.g;
    const int t = threadIdx.x, vec = t % g.V, prow = t / g.V;
    const int64_t image = at.image, per_tile = (int64_t)g.P * g.k, first = at.tile * per_tile;
    const int64_t rows = min(per_tile, p.pixels - first);
    const int left = (int)(rows - prow);
    const int64_t start = ((image * p.pixels + first + prow) * p.C + at.c0) * T::SIZE, step = (int64_t)g.P * p.C * T::SIZE;
    Row<T, 8, TAIL> raw[K];
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (i < g.k) raw[i].load((const char *)p.x + start + i * step, vec, g.V, at.w, i * g.P < left);
    Coef<TAIL, NV> cf;
    load_vec<8, TAIL>(p.w ? p.w + at.c0 : nullptr, 1.f, vec, g.V, at.w, cf.a);
    load_vec<8, TAIL>(p.b ? p.b + at.c0 : nullptr, 0.f, vec, g.V, at.w, cf.b);
    // A wave a group, its lanes the tiles: the mean by its distance from the first tile's, then M2
    const int lane = t & 63, waves = blockDim.x >> 6;   // (whole ones, at least one)
    const float last = (float)(p.pixels - (g.tiles - 1) * per_tile), all = (float)p.pixels;
    if (t >> 6 < waves)
        for (int j = t >> 6; j < at.ngl; j += waves) {
            const float *part = p.part + (image * g.tiles * p.G + at.chunk * g.ng + j) * 2;
            const float m0 = part[0];
            float d = 0.f, m2 = 0.f;
            for (int i = lane; i < g.tiles; i += 64)
                d = fmaf((i + 1 < g.tiles ? (float)per_tile : last) / all, part[(int64_t)i * p.G * 2] - m0, d);
            const float mean = m0 + wave_sum(d);
            for (int i = lane; i < g.tiles; i += 64) {
                const f32x2 q = *(const f32x2 *)(part + (int64_t)i * p.G * 2);
                const float e = q[0] - mean;
                m2 += q[1] + e * e * ((i + 1 < g.tiles ? (float)per_tile : last) * (float)p.cpg);
            }
            const float inv = 1.f / sqrtf(wave_sum(m2) / (all * (float)p.cpg) + p.eps);
            if (lane == 0) {
                lds[2 * j] = mean;
                lds[2 * j + 1] = inv;
                if (at.tile == 0 && p.stats) *(f32x2 *)(p.stats + (image * p.G + at.chunk * g.ng + j) * 2) = f32x2{mean, inv};
            }
        }
    int gi[NV];
    groups_of<NV>(vec, p.cpg, at.ngl, gi);
    __syncthreads();
#pragma unroll
    for (int e = 0; e < NV; ++e) cf.mean[e] = lds[2 * gi[e]];
#pragma unroll
    for (int e = 0; e < 8; ++e) cf.a[e] *= lds[2 * gi[NV == 1 ? 0 : e] + 1];
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (i < g.k) {
            float v[8];
            raw[i].get(v, vec, g.V, at.w);
            cf.apply(v, p.act);
            if (i * g.P < left) Row<T, 8, TAIL>::store((char *)p.out + start + i * step, vec, g.V, at.w, v);
        }
}

template <typename T, Tail TAIL, int NV, int K>
hipError_t launch_k(const GroupNormArgs &a, hipStream_t st)
{
    const Geo &g = a.g;
    const uint32_t grid = (uint32_t)((a.images + g.ipw - 1) / g.ipw * g.tiles * g.chunks);
    const int lds = lds_floats(g, NV, 1) * (int)sizeof(float), threads = g.V * g.P * g.ipw;
    if (g.tiles == 1) {
        auto k = gn_fwd_kernel<T, TAIL, NV, K, false>;
        const hipError_t e = raise_lds_limit((const void *)k, lds);
        if (e != hipSuccess) return e;
        return launch(k, dim3(grid), dim3(threads), lds, st, nullptr, nullptr, a);
    }
    auto k = gn_fwd_kernel<T, TAIL, NV, K, true>;
    hipError_t e = raise_lds_limit((const void *)k, lds);
    if (e == hipSuccess) e = launch(k, dim3(grid), dim3(threads), lds, st, nullptr, nullptr, a);
    if (e != hipSuccess) return e;
    return launch(gn_fwd_apply_kernel<T, TAIL, NV, K>, dim3(grid), dim3(threads), 2 * g.ng * (int)sizeof(float), st, nullptr, nullptr, a);
}

template <typename T, Tail TAIL, int NV>
hipError_t launch_tail(const GroupNormArgs &a, hipStream_t st)
{
    constexpr int B = 4 / T::SIZE;   // (registers of a vector: 4 B' of 16-bit types, 8 of fp32)
    if (a.g.k <= 2 * B) return launch_k<T, TAIL, NV, 2 * B>(a, st);
    if (a.g.k <= 6 * B) return launch_k<T, TAIL, NV, 6 * B>(a, st);
    return launch_k<T, TAIL, NV, 12 * B>(a, st);
}

template <typename T>
hipError_t launch_type(const GroupNormArgs &a, hipStream_t st)
{
    if (a.cpg % 8 == 0) return launch_tail<T, WHOLE, 1>(a, st);
    if (a.C % 8 == 0 && a.g.ng * a.cpg % 8 == 0) return launch_tail<T, WHOLE, 8>(a, st);
    if (a.C >= 8) return launch_tail<T, PART, 8>(a, st);
    return launch_tail<T, SHORT, 8>(a, st);   // (one chunk)
}

}  // namespace

hipError_t launch_group_norm_fwd(const cbr_group_norm_shape &s, const GroupNormArgs &a, hipStream_t st)
{
    if (s.type == CBR_BF16) return launch_type<Bf16>(a, st);
    if (s.type == CBR_F16) return launch_type<F16>(a, st);
    return launch_type<F32>(a, st);
}

}  // namespace cbr
