// group_norm_bwd.hip -- gradients of the group norm with an activation.  With xhat = (x - mean) inv,
// u = xhat w + b and g = dy act'(u), over an image's pixels S1 = sum g xhat and S0 = sum g of every
// channel, and over a group of M values
//   m0 = sum_c w S0 / M,  m1 = sum_c w S1 / M,  dx = (w g - m0 - xhat m1) inv,
// and over the images dw = sum S1, db = sum S0.  As in the forward a workgroup holds whole groups of
// an image, here of x and dy, in registers, or (large images) one kernel leaves the tiles' S1, S0 and
// a second one reads again.
#include <algorithm>

#include "block_launch.h"
#include "group_norm.h"

namespace cbr {
namespace {

using namespace gnorm;

// With d = x - mean: u = d a + b (SiLU: v = -log2(e) u, see scaled_sigmoid).
template <int NV>
struct Coef {
    float mean[NV], inv[NV], a[8], b[8];
    // of channel e: d, and g = dy act'(u); SCALED: -ln 2 times that for SiLU, so that g times a is w g inv for all
    template <bool SCALED>
    __device__ __forceinline__ void grad(int e, float x, float dy, const Split<NV> &sp, int act, float &d, float &g) const
    {
        d = x - sp.pick(mean, e);
        if (act == CBR_ACT_NONE) {
            g = dy;
        } else {
            const float u = fmaf(d, a[e], b[e]);
            if (act == CBR_ACT_RELU) {
                g = u > 0.f ? dy : u <= 0.f ? 0.f : u;   // a NaN stays one
            } else {
                float power;
                const float s = scaled_sigmoid(u, power);   // -ln 2 sigmoid
                // 1 + u (1 - sigmoid), with u = -ln 2 v: 1 - sigmoid as 2^v sigmoid, which keeps its digits where it is
                // small (the difference from 1 lost them: the slope at 14 was off by 13 half steps).  Past the largest
                // number s is 0.
                const float h = fmaf(u, fminf(power, __FLT_MAX__) * s, 1.f);
                g = dy * (SCALED ? s * h : (-LOG2E * s) * h);
            }
        }
    }
    template <Tail TAIL>
    __device__ __forceinline__ void load(const GroupNormArgs &p, const Place &at, const Thread &me, const Split<NV> &sp)
    {
        load_vec<8, TAIL>(p.w ? p.w + at.c0 : nullptr, 1.f, me.vec, p.g.V, at.w, a);
        load_vec<8, TAIL>(p.b ? p.b + at.c0 : nullptr, 0.f, me.vec, p.g.V, at.w, b);
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            const f32x2 st = me.image < p.images ? *(const f32x2 *)(p.stats_in + (me.image * p.G + at.chunk * p.g.ng + sp.gi[e]) * 2) : f32x2{0.f, 0.f};
            mean[e] = st[0];
            inv[e] = st[1];
        }
        const float c = p.act == CBR_ACT_SILU ? -LOG2E : 1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            a[e] *= sp.pick(inv, e) * c;
            b[e] *= c;
        }
    }
};

// A pixel added to a thread's sums of g d and g for each channel.
template <typename T, int NV>
__device__ __forceinline__ void add_pixel(const Coef<NV> &cf, const Raw8<T> &rx, const Raw8<T> &rd, const Split<NV> &sp, int act, float (&s1)[8], float (&s0)[8])
{
    float x[8], dy[8];
    unpack8<T>(rx, x);
    unpack8<T>(rd, dy);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float d, g;
        cf.template grad<false>(e, x[e], dy[e], sp, act, d, g);
        s0[e] += g;
        s1[e] = fmaf(g, d, s1[e]);
    }
}

// dx of a pixel's eight channels: w g inv - c0 - d c1.
template <typename T, int NV>
__device__ __forceinline__ void dx_of(const Coef<NV> &cf, const Raw8<T> &rx, const Raw8<T> &rd, const Split<NV> &sp, int act, const float (&c1)[NV],
                                      const float (&c0)[NV], float (&x)[8])
{
    float dy[8];
    unpack8<T>(rx, x);
    unpack8<T>(rd, dy);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float d, g;
        cf.template grad<true>(e, x[e], dy[e], sp, act, d, g);
        x[e] = fmaf(g, cf.a[e], fmaf(-sp.pick(c1, e), d, -sp.pick(c0, e)));
    }
}

// A thread's S1 and S0 added within its wave and left in LDS: rows [2][8 V ipw].
__device__ __forceinline__ void leave_channels(const Geo &g, const Thread &me, float (&s1)[8], float (&s0)[8], float *red)
{
    const int wd = 8 * g.V * g.ipw;
    if (g.pre) add_same<8>(s1, s0, g.V);
    const int row = g.pre ? me.prow * g.V / 64 : me.prow, c = (me.sub * g.V + me.vec) * 8;
    if (!g.pre || (threadIdx.x & 63) < (unsigned)g.V)
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            *(f32x4 *)(red + 2 * row * wd + c + e) = f32x4{s1[e], s1[e + 1], s1[e + 2], s1[e + 3]};
            *(f32x4 *)(red + (2 * row + 1) * wd + c + e) = f32x4{s0[e], s0[e + 1], s0[e + 2], s0[e + 3]};
        }
}

// Behind a barrier: the columns' sums in a fixed order; `use` is called with the sum, which of the two it is, the image
// and the channel of the chunk.
template <typename F>
__device__ __forceinline__ void take_channels(const Geo &g, const float *red, F &&use)
{
    const int wd = 8 * g.V * g.ipw, rows = sum_rows(g);
    for (int i = threadIdx.x; i < 2 * wd; i += blockDim.x) {
        float v = 0.f;
        for (int r = 0; r < rows; ++r) v += red[2 * r * wd + i];
        const int s = i >= wd, j = i - s * wd;
        use(v, s, j / (8 * g.V), j % (8 * g.V));
    }
}

// Images held whole: x and dy are read once.  (196 x 256 bf16: 6.4 us, a chain of latencies.)
template <typename T, Tail TAIL, int NV, int K>
__global__ __launch_bounds__(1024) void gn_bwd_kernel(GroupNormArgs p)
{
    extern __shared__ __attribute__((aligned(16))) float lds[];
    const Place at(p);
    const Geo &g = p.g;
    const Thread me(p, at);
    const int row = me.sub * (int)p.pixels + me.prow;
    const Part<T, TAIL> ix(p.x, me.first, row, p.C, g.P, me.vec, at.w), id(p.dy, me.first, row, p.C, g.P, me.vec, at.w);
    Raw8<T> rx[K], rd[K];
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (i < g.k) {
            ix.load(rx[i], i, i * g.P < me.left);
            id.load(rd[i], i, i * g.P < me.left);
        }
    const Split<NV> sp(me.vec, p.cpg, at.ngl);
    Coef<NV> cf;
    cf.template load<TAIL>(p, at, me, sp);
    float *const channels = lds + sum_floats(g, NV, 2);
    float s[2][NV];
    {
        float s1[8] = {}, s0[8] = {};
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (i < g.k && i * g.P < me.left) {
                ix.settle(rx[i]);
                id.settle(rd[i]);
                add_pixel<T, NV>(cf, rx[i], rd[i], sp, p.act, s1, s0);
            }
        // The groups' sums of w g xhat and w g (a is w inv, times SiLU's constant: see below), beside the channels'
        float t1[8], t0[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const bool real = TAIL == WHOLE || 8 * me.vec + e < at.w;
            t1[e] = real ? cf.a[e] * s1[e] : 0.f;
            t0[e] = real ? cf.a[e] * s0[e] : 0.f;
            s1[e] *= sp.pick(cf.inv, e);
        }
        sp.collapse(t1, s[0]);
        sp.collapse(t0, s[1]);
        leave_channels(g, me, s1, s0, channels);
    }
    GroupSum<NV, 2> sum(p, lds, me);
    sum(s, sp);
    if (p.out) {
        const float m = (p.act == CBR_ACT_SILU ? -LN2 : 1.f) / ((float)p.pixels * (float)p.cpg);
        float c1[NV], c0[NV];   // inv^2 mean(w g xhat), inv mean(w g)
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            c1[e] = s[0][e] * m * cf.inv[e] * cf.inv[e];
            c0[e] = s[1][e] * m;
        }
        const Part<T, TAIL> out(p.out, me.first, row, p.C, g.P, me.vec, at.w);
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (i < g.k) {
                float x[8];
                dx_of<T, NV>(cf, rx[i], rd[i], sp, p.act, c1, c0, x);
                out.store(x, i, i * g.P < me.left, p.nt);
            }
    }
    // Beside the stores: a single image's sums are the gradients, others parts of them
    take_channels(g, channels, [&](float v, int i, int im, int ch) __attribute__((always_inline)) {
        if (ch >= at.w || at.image + im >= p.images) return;
        if (p.part) p.part[((at.image + im) * 2 + i) * p.C + at.c0 + ch] = v;
        else if (float *o = i ? p.db : p.dw) o[at.c0 + ch] = v;
    });
}

// A pixel of x and dy.
template <typename T, Tail TAIL>
struct Pair {
    Raw8<T> x, d;
    __device__ __forceinline__ void fetch(const Part<T, TAIL> &ix, const Part<T, TAIL> &id, int i, bool on)
    {
        ix.load(x, i, on);
        id.load(d, i, on);
    }
    __device__ __forceinline__ void settle(const Part<T, TAIL> &ix)
    {
        ix.settle(x);
        ix.settle(d);
    }
};

// First kernel of large images: a tile's S1 and S0 of each channel.  One pixel is on its way while another is added: more
// of them cost waves (four and four, bf16: 64 x 56 x 56 x 256 111 us; two and two 99; one and one 96).
template <typename T, Tail TAIL, int NV>
__global__ __launch_bounds__(1024) void gn_bwd_tiles_kernel(GroupNormArgs p)
{
    extern __shared__ __attribute__((aligned(16))) float lds[];
    const Place at(p);
    const Geo &g = p.g;
    const Thread me(p, at);
    const Part<T, TAIL> ix(p.x, me.first, me.prow, p.C, g.P, me.vec, at.w), id(p.dy, me.first, me.prow, p.C, g.P, me.vec, at.w);
    const Split<NV> sp(me.vec, p.cpg, at.ngl);
    const int own = me.pixels(g);
    Pair<T, TAIL> one, two;
    one.fetch(ix, id, 0, 0 < own);
    Coef<NV> cf;
    cf.template load<TAIL>(p, at, me, sp);
    float s1[8] = {}, s0[8] = {};
    auto add = [&](Pair<T, TAIL> &r, int i) __attribute__((always_inline)) {
        r.settle(ix);
        if (i < own) add_pixel<T, NV>(cf, r.x, r.d, sp, p.act, s1, s0);
    };
    for (int i = 0; i < g.k; i += 2) {
        two.fetch(ix, id, i + 1, i + 1 < own);
        add(one, i);
        one.fetch(ix, id, i + 2, i + 2 < own);
        add(two, i + 1);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s1[e] *= sp.pick(cf.inv, e);
    leave_channels(g, me, s1, s0, lds);
    __syncthreads();
    take_channels(g, lds, [&](float v, int i, int, int ch) __attribute__((always_inline)) {
        if (ch < at.w) p.part[((me.image * g.tiles + at.tile) * 2 + i) * p.C + at.c0 + ch] = v;
    });
}

// dw, db of FC channels a workgroup: the images' and tiles' parts added in fp64, in a fixed order, by rows of FC
// threads (64 channels a workgroup left one to read 2 MB: 12.9 us of 8 x 50176 x 64; 16: 5).  LDS: two doubles a thread.
constexpr int FC = 16;

__device__ __forceinline__ void finish_channels(const GroupNormArgs &p, double *sums)
{
    int lanes = 1;   // rows of threads, a power of two
    while (2 * lanes * FC <= (int)blockDim.x) lanes *= 2;
    const int c = blockIdx.x * FC + (threadIdx.x % FC), lane = threadIdx.x / FC;
    const int64_t rows = p.images * p.g.tiles, ld = 2 * (int64_t)p.C;
    double s1 = 0., s0 = 0.;
    if (c < p.C && lane < lanes) {
        const float *q = p.part + c;
        int64_t r = lane;
        for (; r + 7 * lanes < rows; r += 8 * lanes) {   // sixteen loads under way
            float v[8], w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = q[(r + i * lanes) * ld];
                w[i] = q[(r + i * lanes) * ld + p.C];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s1 += v[i];
                s0 += w[i];
            }
        }
        for (; r < rows; r += lanes) {
            s1 += q[r * ld];
            s0 += q[r * ld + p.C];
        }
    }
    sums[2 * threadIdx.x] = s1;
    sums[2 * threadIdx.x + 1] = s0;
    for (int n = lanes / 2; n > 0; n /= 2) {
        __syncthreads();
        if (lane < n) {
            s1 += sums[2 * (threadIdx.x + n * FC)];
            s0 += sums[2 * (threadIdx.x + n * FC) + 1];
            sums[2 * threadIdx.x] = s1;
            sums[2 * threadIdx.x + 1] = s0;
        }
    }
    if (lane == 0 && c < p.C) {
        if (p.dw) p.dw[c] = (float)s1;
        if (p.db) p.db[c] = (float)s0;
    }
}

__global__ __launch_bounds__(1024) void gn_bwd_finish_kernel(GroupNormArgs p)
{
    extern __shared__ __attribute__((aligned(16))) double sums[];
    finish_channels(p, sums);
}

// Second kernel of large images: the tiles' sums joined, then the tile's dx.  Both are bound by memory: 64 x 56 x 56 x 256
// bf16 36 + 51 us for two and three passes over 103 MB, 5.7 and 6.0 TB/s with what is left in the caches.  LDS (floats): [parts][2][8 V] sums of some
// tiles, [2][8 V] columns, [2][ng] groups.  The first `front` workgroups add up dw and db beside it (a
// kernel of its own behind this one took 2 to 3 us more: 64 x 56 x 56 x 256 110 us against 108, 2 x 4097 x 64 17.8, 16.1).
inline __host__ __device__ int apply_parts(const Geo &g) { return max(1, min(g.V * g.P / (16 * g.V), 8)); }
inline int apply_floats(const Geo &g) { return 16 * g.V * (apply_parts(g) + 1) + 2 * g.ng; }

template <typename T, Tail TAIL, int NV>
__global__ __launch_bounds__(1024) void gn_bwd_apply_kernel(GroupNormArgs p)
{
    extern __shared__ __attribute__((aligned(16))) float lds[];
    if (blockIdx.x < (uint32_t)p.front) {
        finish_channels(p, (double *)lds);
        return;
    }
    const Place at(p);
    const Geo &g = p.g;
    const Thread me(p, at);
    const Part<T, TAIL> ix(p.x, me.first, me.prow, p.C, g.P, me.vec, at.w), id(p.dy, me.first, me.prow, p.C, g.P, me.vec, at.w),
        out(p.out, me.first, me.prow, p.C, g.P, me.vec, at.w);
    const int own = me.pixels(g);
    Pair<T, TAIL> one, two;
    one.fetch(ix, id, 0, 0 < own);
    const Split<NV> sp(me.vec, p.cpg, at.ngl);
    Coef<NV> cf;
    cf.template load<TAIL>(p, at, me, sp);
    // The tiles' sums of the chunk's channels, added in a fixed order by some threads a channel
    const int t = threadIdx.x, wd = 8 * g.V, parts = apply_parts(g);
    float *const red = lds, *const col = red + 2 * wd * parts, *const tot = col + 2 * wd;
    for (int i = t; i < 2 * wd * parts; i += blockDim.x) {
        const int c = i % (2 * wd), s = c >= wd, ch = c - s * wd;
        float v = 0.f;
        if (ch < at.w) {
            const float *q = p.part + (me.image * g.tiles * 2 + s) * p.C + at.c0 + ch;
            const int64_t ld = 2 * (int64_t)p.C;
            int r = i / (2 * wd);
            for (; r + 7 * parts < g.tiles; r += 8 * parts) {   // eight loads under way
                float w[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) w[u] = q[(r + u * parts) * ld];
#pragma unroll
                for (int u = 0; u < 8; ++u) v += w[u];
            }
            for (; r < g.tiles; r += parts) v += q[r * ld];
        }
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
    columns_to_groups<8>(col, tot, p.cpg, wd, at.ngl, 1);
    columns_to_groups<8>(col + wd, tot + g.ng, p.cpg, wd, at.ngl, 1);
    __syncthreads();
    const float m = 1.f / ((float)p.pixels * (float)p.cpg);
    float c1[NV], c0[NV];
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        c1[e] = tot[sp.gi[e]] * m * cf.inv[e] * cf.inv[e];
        c0[e] = tot[g.ng + sp.gi[e]] * m * cf.inv[e];
    }
    auto finish = [&](Pair<T, TAIL> &r, int i) __attribute__((always_inline)) {
        float x[8];
        r.settle(ix);
        dx_of<T, NV>(cf, r.x, r.d, sp, p.act, c1, c0, x);
        out.store(x, i, i < own, p.nt);
    };
    for (int i = 0; i < g.k; i += 2) {
        two.fetch(ix, id, i + 1, i + 1 < own);
        finish(one, i);
        one.fetch(ix, id, i + 2, i + 2 < own);
        finish(two, i + 1);
    }
}

template <typename Kern>
hipError_t launch_with(Kern k, const GroupNormArgs &a, int lds, hipStream_t st)
{
    const Geo &g = a.g;
    const uint32_t grid = (uint32_t)((a.images + g.ipw - 1) / g.ipw * g.tiles * g.chunks) + a.front;
    const hipError_t e = raise_lds_limit((const void *)k, lds);
    if (e != hipSuccess) return e;
    return launch(k, dim3(grid), dim3(threads_of(g)), lds, st, nullptr, nullptr, a);
}

template <typename T, Tail TAIL, int NV>
hipError_t launch_tail(const GroupNormArgs &a, hipStream_t st)
{
    constexpr int B = 4 / T::SIZE;
    const Geo &g = a.g;
    const int lds = bwd_floats(g, a.cpg) * (int)sizeof(float), fin = a.part && (a.dw || a.db) ? (a.C + FC - 1) / FC : 0;
    hipError_t e;
    if (g.tiles > 1) {
        e = launch_with(gn_bwd_tiles_kernel<T, TAIL, NV>, a, lds, st);
        if (e != hipSuccess) return e;
        if (a.out) {
            GroupNormArgs b = a;
            b.front = fin;
            return launch_with(gn_bwd_apply_kernel<T, TAIL, NV>, b, std::max(apply_floats(g) * (int)sizeof(float), fin ? threads_of(g) * 16 : 0), st);
        }
    } else if (g.k <= B) {
        e = launch_with(gn_bwd_kernel<T, TAIL, NV, B>, a, lds, st);
    } else if (g.k <= 2 * B) {
        e = launch_with(gn_bwd_kernel<T, TAIL, NV, 2 * B>, a, lds, st);
    } else {
        e = launch_with(gn_bwd_kernel<T, TAIL, NV, bwd_most(NV) * B>, a, lds, st);
    }
    if (e != hipSuccess || !fin) return e;
    return launch(gn_bwd_finish_kernel, dim3(fin), dim3(1024), 1024 * 16, st, nullptr, nullptr, a);
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

hipError_t launch_group_norm_bwd(const cbr_group_norm_shape &s, const GroupNormArgs &a, hipStream_t st)
{
    if (s.type == CBR_BF16) return launch_type<Bf16>(a, st);
    if (s.type == CBR_F16) return launch_type<F16>(a, st);
    return launch_type<F32>(a, st);
}

}  // namespace cbr
