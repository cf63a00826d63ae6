// group_norm_bwd.hip -- gradients of the group norm with an activation.  With xhat = (x - mean) inv,
// u = xhat w + b and g = dy act'(u), over an image's pixels S1 = sum g xhat and S0 = sum g of every
// channel, and over a group of M values
//   m0 = sum_c w S0 / M,  m1 = sum_c w S1 / M,  dx = (w g - m0 - xhat m1) inv,
// and over the images dw = sum S1, db = sum S0.  As in the forward a workgroup holds whole groups of
// an image, here of x and dy, in registers, or (large images) one kernel leaves the tiles' S1, S0 and
// a second one reads again.
#include "block_launch.h"
#include "group_norm.h"

namespace cbr {
namespace {

using namespace gnorm;

template <int NV>
struct Coef {
    float mean[NV], inv[NV], w[8], b[8];
    // of channel e: xhat, and g = dy act'(u)
    __device__ __forceinline__ void grad(int e, float x, float dy, int act, float &xhat, float &g) const
    {
        const int s = NV == 1 ? 0 : e;
        xhat = (x - mean[s]) * inv[s];
        if (act == CBR_ACT_NONE) {
            g = dy;
        } else {
            const float u = fmaf(xhat, w[e], b[e]);
            if (act == CBR_ACT_RELU) {
                g = u > 0.f ? dy : u <= 0.f ? 0.f : u;   // a NaN stays one
            } else {
                const float y = sigmoid(u);
                g = dy * (y * fmaf(u, 1.f - y, 1.f));
            }
        }
    }
};

// TILES: leaves the tile's S1 and S0 of each channel; else also dx.
template <typename T, Tail TAIL, int NV, int K, bool TILES>
__global__ __launch_bounds__(1024) void gn_bwd_kernel(GroupNormArgs p)
{
    extern __shared__ __attribute__((aligned(16))) float lds[];
    const Place<false> at(p, gridDim.x);
    const Geo &g = p.g;
    const int t = threadIdx.x, vec = t % g.V, q = t / g.V, prow = q % g.P, sub = q / g.P;
    const int64_t image = at.image + sub, first = (int64_t)at.tile * g.P * g.k;
    const int64_t rows = min((int64_t)g.P * g.k, p.pixels - first);
    const bool on = image < p.images;
    const int left = (int)(rows - prow);
    const int64_t start = ((image * p.pixels + first + prow) * p.C + at.c0) * T::SIZE, step = (int64_t)g.P * p.C * T::SIZE;
    Row<T, 8, TAIL> rx[K], rd[K];
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (i < g.k) {
            rx[i].load((const char *)p.x + start + i * step, vec, g.V, at.w, on && i * g.P < left);
            rd[i].load((const char *)p.dy + start + i * step, vec, g.V, at.w, on && i * g.P < left);
        }
    Coef<NV> cf;
    load_vec<8, TAIL>(p.w ? p.w + at.c0 : nullptr, 1.f, vec, g.V, at.w, cf.w);
    load_vec<8, TAIL>(p.b ? p.b + at.c0 : nullptr, 0.f, vec, g.V, at.w, cf.b);
    int gi[NV];
    groups_of<NV>(vec, p.cpg, at.ngl, gi);
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        const f32x2 st = on ? *(const f32x2 *)(p.stats_in + (image * p.G + at.chunk * g.ng + gi[e]) * 2) : f32x2{0.f, 0.f};
        cf.mean[e] = st[0];
        cf.inv[e] = st[1];
    }
    float s1[8] = {}, s0[8] = {};
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (i < g.k && i * g.P < left) {
            float x[8], d[8];
            rx[i].get(x, vec, g.V, at.w);
            rd[i].get(d, vec, g.V, at.w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float xhat, gr;
                cf.grad(e, x[e], d[e], p.act, xhat, gr);
                s0[e] += gr;
                s1[e] = fmaf(gr, xhat, s1[e]);
            }
        }
    // Over the pixels: within the waves, then through LDS in a fixed order
    const int wd = 8 * g.V * g.ipw, nrows = g.pre ? g.P * g.V / 64 : g.P;
    float *const red = lds, *const col = red + 2 * nrows * wd, *const tot = col + 2 * wd;   // [2] of each
    {
        if (g.pre) add_same<8>(s1, s0, g.V);
        const int row = g.pre ? prow * g.V / 64 : prow, c = (sub * g.V + vec) * 8;
        if (!g.pre || (t & 63) < g.V)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                red[2 * row * wd + c + e] = s1[e];
                red[(2 * row + 1) * wd + c + e] = s0[e];
            }
    }
    __syncthreads();
    for (int c = t; c < 2 * wd; c += blockDim.x) {
        float v = 0.f;
        for (int r = 0; r < nrows; ++r) v += red[2 * r * wd + c];
        // column c of a sum: image c / (8 V), channel c % (8 V) of the chunk
        const int s = c >= wd, cc = c - s * wd, im = cc / (8 * g.V), ch = cc % (8 * g.V);
        if (ch < at.w && at.image + im < p.images) {
            // one image and one tile: these are the gradients; else parts of them
            if (p.part) p.part[(((at.image + im) * g.tiles + at.tile) * 2 + s) * p.C + at.c0 + ch] = v;
            else if (float *o = s ? p.db : p.dw) o[at.c0 + ch] = v;
            if constexpr (!TILES) col[c] = v * (p.w ? p.w[at.c0 + ch] : 1.f);
        }
    }
    if constexpr (!TILES) {
        if (!p.out) return;
        __syncthreads();
        columns_to_groups(col, tot, p.cpg, 8 * g.V, g.ng, g.ipw);
        columns_to_groups(col + wd, tot + g.ng * g.ipw, p.cpg, 8 * g.V, g.ng, g.ipw);
        __syncthreads();
        const float m = 1.f / ((float)p.pixels * (float)p.cpg);
        float m1[NV], m0[NV];
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            m1[e] = tot[sub * g.ng + gi[e]] * m;
            m0[e] = tot[g.ng * g.ipw + sub * g.ng + gi[e]] * m;
        }
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (i < g.k && on && i * g.P < left) {
                float x[8], d[8];
                rx[i].get(x, vec, g.V, at.w);
                rd[i].get(d, vec, g.V, at.w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float xhat, gr;
                    const int z = NV == 1 ? 0 : e;
                    cf.grad(e, x[e], d[e], p.act, xhat, gr);
                    x[e] = (fmaf(gr, cf.w[e], -m0[z]) - xhat * m1[z]) * cf.inv[z];
                }
                Row<T, 8, TAIL>::store((char *)p.out + start + i * step, vec, g.V, at.w, x);
            }
    }
}

// dw, db of 64 channels from c0 on: the images' and tiles' parts added in fp64, in a fixed order.
__device__ __forceinline__ void finish(const GroupNormArgs &p, int c0, double *lds)
{
    const int c = c0 + (threadIdx.x & 63), wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int64_t rows = p.images * p.g.tiles;
    double s1 = 0., s0 = 0.;
    if (c < p.C && wave < waves)
        for (int64_t r = wave; r < rows; r += waves) {
            s1 += p.part[2 * r * p.C + c];
            s0 += p.part[(2 * r + 1) * p.C + c];
        }
    lds[2 * threadIdx.x] = s1;
    lds[2 * threadIdx.x + 1] = s0;
    __syncthreads();
    if (threadIdx.x < 64 && c < p.C) {
        for (int i = 1; i < waves; ++i) {
            s1 += lds[2 * (threadIdx.x + 64 * i)];
            s0 += lds[2 * (threadIdx.x + 64 * i) + 1];
        }
        if (p.dw) p.dw[c] = (float)s1;
        if (p.db) p.db[c] = (float)s0;
    }
}

__global__ __launch_bounds__(1024) void gn_bwd_finish_kernel(GroupNormArgs p)
{
    extern __shared__ __attribute__((aligned(16))) float lds[];
    finish(p, blockIdx.x * 64, (double *)lds);
}

// Second kernel of large images: the tiles' sums joined, then the tile's dx.
template <typename T, Tail TAIL, int NV, int K>
__global__ __launch_bounds__(1024) void gn_bwd_apply_kernel(GroupNormArgs p)
{
    extern __shared__ __attribute__((aligned(16))) float lds[];
    const Geo &g = p.g;
    const Place<true> at(p, gridDim.x);
    const int t = threadIdx.x, vec = t % g.V, prow = t / g.V;
    const int64_t image = at.image, per_tile = (int64_t)g.P * g.k, first = at.tile * per_tile;
    const int64_t rows = min(per_tile, p.pixels - first);
    const int left = (int)(rows - prow);
    const int64_t start = ((image * p.pixels + first + prow) * p.C + at.c0) * T::SIZE, step = (int64_t)g.P * p.C * T::SIZE;
    Row<T, 8, TAIL> rx[K], rd[K];
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (i < g.k) {
            rx[i].load((const char *)p.x + start + i * step, vec, g.V, at.w, i * g.P < left);
            rd[i].load((const char *)p.dy + start + i * step, vec, g.V, at.w, i * g.P < left);
        }
    Coef<NV> cf;
    load_vec<8, TAIL>(p.w ? p.w + at.c0 : nullptr, 1.f, vec, g.V, at.w, cf.w);
    load_vec<8, TAIL>(p.b ? p.b + at.c0 : nullptr, 0.f, vec, g.V, at.w, cf.b);
    int gi[NV];
    groups_of<NV>(vec, p.cpg, at.ngl, gi);
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        const f32x2 st = *(const f32x2 *)(p.stats_in + (image * p.G + at.chunk * g.ng + gi[e]) * 2);
        cf.mean[e] = st[0];
        cf.inv[e] = st[1];
    }
    // The tiles' sums of the chunk's channels, added in a fixed order by some threads a channel
    const int wd = 8 * g.V, parts = max(1, min((int)blockDim.x / (2 * wd), 8));
    float *const red = lds, *const col = red + 2 * wd * parts, *const tot = col + 2 * wd;
    for (int i = t; i < 2 * wd * parts; i += blockDim.x) {
        const int c = i % (2 * wd), s = c >= wd, ch = c - s * wd;
        float v = 0.f;
        if (ch < at.w)
            for (int r = i / (2 * wd); r < g.tiles; r += parts)
                v += p.part[((image * g.tiles + r) * 2 + s) * p.C + at.c0 + ch];
        red[i] = v;
    }
    __syncthreads();
    for (int c = t; c < 2 * wd; c += blockDim.x) {
        const int ch = c % wd;
        float v = 0.f;
        for (int r = 0; r < parts; ++r) v += red[r * 2 * wd + c];
        if (ch < at.w) col[c] = v * (p.w ? p.w[at.c0 + ch] : 1.f);
    }
    __syncthreads();
    columns_to_groups(col, tot, p.cpg, wd, g.ng, 1);
    columns_to_groups(col + wd, tot + g.ng, p.cpg, wd, g.ng, 1);
    __syncthreads();
    const float m = 1.f / ((float)p.pixels * (float)p.cpg);
    float m1[NV], m0[NV];
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        m1[e] = tot[gi[e]] * m;
        m0[e] = tot[g.ng + gi[e]] * m;
    }
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (i < g.k && i * g.P < left) {
            float x[8], d[8];
            rx[i].get(x, vec, g.V, at.w);
            rd[i].get(d, vec, g.V, at.w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float xhat, gr;
                const int z = NV == 1 ? 0 : e;
                cf.grad(e, x[e], d[e], p.act, xhat, gr);
                x[e] = (fmaf(gr, cf.w[e], -m0[z]) - xhat * m1[z]) * cf.inv[z];
            }
            Row<T, 8, TAIL>::store((char *)p.out + start + i * step, vec, g.V, at.w, x);
        }
}

template <typename T, Tail TAIL, int NV, int K>
hipError_t launch_k(const GroupNormArgs &a, hipStream_t st)
{
    const Geo &g = a.g;
    const uint32_t grid = (uint32_t)((a.images + g.ipw - 1) / g.ipw * g.tiles * g.chunks);
    const int lds = lds_floats(g, 8, 2) * (int)sizeof(float), threads = g.V * g.P * g.ipw;
    auto k = g.tiles == 1 ? gn_bwd_kernel<T, TAIL, NV, K, false> : gn_bwd_kernel<T, TAIL, NV, K, true>;
    hipError_t e = raise_lds_limit((const void *)k, lds);
    if (e == hipSuccess) e = launch(k, dim3(grid), dim3(threads), lds, st, nullptr, nullptr, a);
    if (e != hipSuccess) return e;
    if (g.tiles > 1 && a.out) {
        auto k2 = gn_bwd_apply_kernel<T, TAIL, NV, K>;
        const int wd = 8 * g.V, parts = std::max(1, std::min(threads / (2 * wd), 8));
        const int lds2 = (2 * wd * (parts + 1) + 2 * g.ng) * (int)sizeof(float);
        e = raise_lds_limit((const void *)k2, lds2);
        if (e == hipSuccess) e = launch(k2, dim3(grid), dim3(threads), lds2, st, nullptr, nullptr, a);
        if (e != hipSuccess) return e;
    }
    if (a.part && (a.dw || a.db)) {
        const int n = a.images * g.tiles >= 64 ? 1024 : 256;
        return launch(gn_bwd_finish_kernel, dim3((a.C + 63) / 64), dim3(n), n * 16, st, nullptr, nullptr, a);
    }
    return hipSuccess;
}

template <typename T, Tail TAIL, int NV>
hipError_t launch_tail(const GroupNormArgs &a, hipStream_t st)
{
    constexpr int B = 4 / T::SIZE;
    if (a.g.k <= B) return launch_k<T, TAIL, NV, B>(a, st);
    if (a.g.k <= 3 * B) return launch_k<T, TAIL, NV, 3 * B>(a, st);
    return launch_k<T, TAIL, NV, 6 * B>(a, st);
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

hipError_t launch_group_norm_bwd(const cbr_group_norm_shape &s, const GroupNormArgs &a, hipStream_t st)
{
    if (s.type == CBR_BF16) return launch_type<Bf16>(a, st);
    if (s.type == CBR_F16) return launch_type<F16>(a, st);
    return launch_type<F32>(a, st);
}

}  // namespace cbr
