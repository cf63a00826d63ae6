// block_norm_bwd.hip -- backward of the residual add around a block with the norms on both
// its sides (n = post(f), y = x + alpha r g n, h = pre(y)), in one pass over dy, dh, y, f:
//   D   = dy + is' (dh w' - mean(dh w') - yhat mean(dh w' yhat)),     dx = D
//   u   = alpha r g D,   df = is (u w - mean(u w) - nhat mean(u w nhat))
// (means over the channels of a row; the middle term only for a layer norm), and two sums
// over rows for each norm, from which every parameter's gradient follows:
//   S1 = sum D nhat, S0 = sum D  (of one gate row):  dg = alpha r (w S1 + b S0),
//   dr = alpha sum_i g_i (w S1_i + b S0_i), dw = alpha r sum_i g_i S1_i, db = alpha r sum_i g_i S0_i
//   T1 = sum dh yhat, T0 = sum dh:  dw' = T1, db' = T0.
// The sums stay in registers over a workgroup's rows and leave as one partial row; a second
// kernel adds the partial rows in fp64.
#include "block_norm.h"

namespace cbr {
namespace {

using namespace bnorm;

// How the rows are dealt out.  SPLIT: a gate row's rows go to `per` workgroups, each within
// one gate row, and the partial sums are S1, S0, T1, T0 of that gate row.  Otherwise every
// group of L threads owns `gates` whole gate rows: it finishes their dgate itself and the
// partial sums are sum g S1, sum g S0, T1, T0.
struct Deal {
    int blocks, per, gates;
    bool split;
};

constexpr int BWD_THREADS = 512;
// Workgroups at most: two of 512 threads fit a CU's registers at a time (a partial row is 16
// bytes a channel written and read again, so more workgroups than run at once only add bytes).
constexpr int BWD_BLOCKS = 512;

Deal deal_of(uint32_t rows, uint32_t rpg, bool gate, const Layout &o)
{
    const uint64_t gates = gate ? rows / rpg : 1;
    if (!gate) rpg = rows;
    auto up = [](uint64_t a, uint64_t b) { return (a + b - 1) / b; };
    const uint64_t subs = (uint64_t)BWD_BLOCKS * o.rpb;
    // rows in turn of the busiest group of threads, either way
    const uint64_t per = std::max<uint64_t>(1, std::min<uint64_t>(BWD_BLOCKS / gates, rpg / (2u * o.rpb)));
    const uint64_t split_turns = up(gates * per, BWD_BLOCKS) * up(up(rpg, per), o.rpb);
    const uint64_t whole_turns = up(gates, subs) * rpg;
    Deal d;
    d.split = !gate || split_turns < whole_turns;
    if (d.split) {
        d.per = (int)per;
        d.gates = 1;
        d.blocks = (int)(gates * per);
    } else {
        d.per = 1;
        d.gates = (int)up(gates, subs);
        d.blocks = (int)up(up(gates, d.gates), o.rpb);
    }
    return d;
}

template <typename TS, typename TB, int E, bool TAIL, bool SPLIT>
__global__ __launch_bounds__(BWD_THREADS) void block_norm_bwd_kernel(BlockNormArgs p, int L, int rpb, int per, int gates)
{
    __shared__ float red[2][MAX_WAVES][2];
    __shared__ float comb[BWD_THREADS * E];
    RowSum<2> sum{red, L, 0};
    const int C = p.C, l = threadIdx.x % L, sub = threadIdx.x / L;
    const bool hasf = p.f != nullptr, haspre = p.pre != CBR_NORM_NONE, haspost = p.post != CBR_NORM_NONE;

    // This thread group's rows: r0 + t * step for t < turns, those below r1 existing.
    uint64_t r0, r1;
    uint32_t step, turns;
    if constexpr (SPLIT) {
        const uint32_t gi = blockIdx.x / per, part = blockIdx.x % per;
        const uint64_t first = (uint64_t)gi * p.rpg;
        const uint64_t a = first + (uint64_t)p.rpg * part / per, b = first + (uint64_t)p.rpg * (part + 1) / per;
        r0 = a + sub;
        r1 = b;
        step = rpb;
        turns = (uint32_t)((b - a + rpb - 1) / rpb);
    } else {
        const uint64_t own = (uint64_t)gates * p.rpg;
        r0 = ((uint64_t)blockIdx.x * rpb + sub) * own;
        r1 = r0 + own < p.rows ? r0 + own : p.rows;
        step = 1;
        turns = (uint32_t)own;
    }

    float ar[E], w[E], pw[E];        // alpha r (SPLIT: alpha r g), post_w, pre_w
    load_vec<E, TAIL>(p.res_scale, 1.f, l, L, C, ar);
    load_vec<E, TAIL>(p.post_w, 1.f, l, L, C, w);
    load_vec<E, TAIL>(p.pre_w, 1.f, l, L, C, pw);
#pragma unroll
    for (int j = 0; j < E; ++j) ar[j] *= p.alpha;
    Row<TB, E, TAIL> graw;
    if constexpr (SPLIT) {
        if (p.gate) {
            float gv[E];
            graw.load((const char *)p.gate + (uint64_t)(blockIdx.x / per) * C * TB::SIZE, l, L, C, true);
            graw.get(gv);
#pragma unroll
            for (int j = 0; j < E; ++j) ar[j] *= gv[j];
        }
    }
    float s1[E], s0[E], t1[E], t0[E], g1[SPLIT ? 1 : E], g0[SPLIT ? 1 : E];
#pragma unroll
    for (int j = 0; j < E; ++j) s1[j] = s0[j] = t1[j] = t0[j] = 0.f;
    if constexpr (!SPLIT)
#pragma unroll
        for (int j = 0; j < E; ++j) g1[j] = g0[j] = 0.f;

    Row<TS, E, TAIL> dyn, yn;
    Row<TB, E, TAIL> dhn, fn;
    f32x2 psn = {0.f, 0.f}, qsn = {0.f, 0.f};
    auto fetch = [&](uint64_t row) __attribute__((always_inline)) {
        const bool on = row < r1;
        dyn.load((const char *)p.dy + row * C * TS::SIZE, l, L, C, on && p.dy);
        yn.load((const char *)p.x + row * C * TS::SIZE, l, L, C, on && haspre);
        dhn.load((const char *)p.dh + row * C * TB::SIZE, l, L, C, on && haspre);
        fn.load((const char *)p.f + row * C * TB::SIZE, l, L, C, on && hasf);
        if (on && haspre) psn = *(const f32x2 *)(p.pre_stats + 2 * row);
        if (on && haspost) qsn = *(const f32x2 *)(p.post_stats + 2 * row);
    };
    // The next row's loads run beside this row's sums; with sixteen values a thread there are
    // no registers for that (90 to 330 spilled), so a row is loaded when its turn comes.
    constexpr bool AHEAD = E == 8;
    if constexpr (AHEAD) fetch(r0);
    uint32_t left = p.rpg;   // rows left of the current gate row (!SPLIT)
    for (uint32_t t = 0; t < turns; ++t) {
        const uint64_t row = r0 + (uint64_t)t * step;
        const bool on = row < r1;
        if constexpr (!AHEAD) fetch(row);
        float d[E], a[E], b[E], f[E];
        dyn.get(d);
        yn.get(a);
        dhn.get(b);
        fn.get(f);
        const f32x2 ps = psn, qs = qsn;
        if constexpr (!SPLIT)
            if (p.gate && left == p.rpg)
                graw.load((const char *)p.gate + (uint64_t)((uint32_t)row / p.rpg) * C * TB::SIZE, l, L, C, on);
        if constexpr (AHEAD)
            if (t + 1 < turns) fetch(row + step);
        if (haspre) {
            float m[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < E; ++j) {
                a[j] = has<E, TAIL>(j, l, L, C) && on ? (a[j] - ps.x) * ps.y : 0.f;   // yhat
                t1[j] = fmaf(b[j], a[j], t1[j]);
                t0[j] += b[j];
                b[j] *= pw[j];
                m[0] = fmaf(b[j], a[j], m[0]);
                m[1] += b[j];
            }
            sum(m);
            const float m1 = m[0] / (float)C, m0 = p.pre == CBR_NORM_LAYER ? m[1] / (float)C : 0.f;
#pragma unroll
            for (int j = 0; j < E; ++j) d[j] = fmaf(b[j] - m0 - a[j] * m1, ps.y, d[j]);
        }
        if (on) Row<TS, E, TAIL>::store((char *)p.dx + row * C * TS::SIZE, l, L, C, d);
        if (hasf) {
            float m[2] = {0.f, 0.f};
            float g[SPLIT ? 1 : E];
            if constexpr (!SPLIT) {
                if (p.gate) graw.get(g);
                else
#pragma unroll
                    for (int j = 0; j < E; ++j) g[j] = 1.f;
            }
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const bool in = has<E, TAIL>(j, l, L, C) && on;
                if (!in) d[j] = 0.f;                                   // rows and channels that do not exist
                if (haspost) f[j] = in ? (f[j] - qs.x) * qs.y : 0.f;   // nhat
                s1[j] = fmaf(d[j], f[j], s1[j]);
                s0[j] += d[j];
                d[j] *= ar[j];
                if constexpr (!SPLIT) d[j] *= g[j];
                if (haspost) {
                    d[j] *= w[j];
                    m[0] = fmaf(d[j], f[j], m[0]);
                    m[1] += d[j];
                }
            }
            if (haspost) {
                sum(m);
                const float m1 = m[0] / (float)C, m0 = p.post == CBR_NORM_LAYER ? m[1] / (float)C : 0.f;
#pragma unroll
                for (int j = 0; j < E; ++j) d[j] = (d[j] - m0 - f[j] * m1) * qs.y;
            }
            if (on) Row<TB, E, TAIL>::store((char *)p.df + row * C * TB::SIZE, l, L, C, d);
            if constexpr (!SPLIT) {
                if (--left == 0) {   // the gate row is done
                    left = p.rpg;
                    if (on && p.dgate) {
                        float pb[E], o[E];
                        load_vec<E, TAIL>(p.post_b, 0.f, l, L, C, pb);
#pragma unroll
                        for (int j = 0; j < E; ++j) o[j] = ar[j] * fmaf(w[j], s1[j], pb[j] * s0[j]);
                        Row<TB, E, TAIL>::store((char *)p.dgate + (uint64_t)((uint32_t)row / p.rpg) * C * TB::SIZE, l,
                                               L, C, o);
                    }
#pragma unroll
                    for (int j = 0; j < E; ++j) {
                        g1[j] = fmaf(g[j], s1[j], g1[j]);
                        g0[j] = fmaf(g[j], s0[j], g0[j]);
                        s1[j] = s0[j] = 0.f;
                    }
                }
            }
        }
    }
    if (!p.part) return;
    // the workgroup's row groups, added in order, one quantity at a time
    for (int q = 0; q < 4; ++q) {
        if (q < 2 ? !hasf : !haspre) continue;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < E; ++j) {
            float v;
            if constexpr (SPLIT) v = q == 0 ? s1[j] : q == 1 ? s0[j] : q == 2 ? t1[j] : t0[j];
            else v = q == 0 ? g1[j] : q == 1 ? g0[j] : q == 2 ? t1[j] : t0[j];
            const int c = col_of<E>(j, l, L);
            comb[sub * L * E + c] = v;
        }
        __syncthreads();
        for (int c = threadIdx.x; c < C; c += blockDim.x) {
            float v = comb[c];
            for (int s = 1; s < rpb; ++s) v += comb[s * L * E + c];
            p.part[((size_t)blockIdx.x * 4 + q) * C + c] = v;
        }
    }
}

// The parameters' gradients from the partial rows, in fp64 and a fixed order.  Blocks
// 0 .. nparam - 1 take 16 channels each: 64 threads a channel over the partial rows, added
// through LDS.  The blocks after them (dgate of a split gate row): 256 channels of one gate
// row each, a thread a channel.
constexpr int FIN_CH = 16, FIN_RG = 64, FIN_THREADS = FIN_CH * FIN_RG;

template <typename TB>
__global__ __launch_bounds__(FIN_THREADS) void block_norm_bwd_finish_kernel(BlockNormArgs p, int blocks, int per,
                                                                            int split, int nparam)
{
    __shared__ double red[4][FIN_RG][FIN_CH];
    const int C = p.C;
    if ((int)blockIdx.x >= nparam) {
        const int tiles = (C + 255) / 256, b = blockIdx.x - nparam;
        const int gi = b / tiles, c = b % tiles * 256 + threadIdx.x;
        if (threadIdx.x >= 256 || c >= C) return;
        double s1 = 0., s0 = 0.;
        for (int k = 0; k < per; ++k) {
            const float *row = p.part + ((size_t)gi * per + k) * 4 * C + c;
            s1 += row[0];
            s0 += row[C];
        }
        const double w = p.post_w ? p.post_w[c] : 1.0, pb = p.post_b ? p.post_b[c] : 0.0;
        const double ar = (double)p.alpha * (p.res_scale ? p.res_scale[c] : 1.0);
        store_one<TB>((char *)p.dgate + ((size_t)gi * C + c) * TB::SIZE, (float)(ar * (w * s1 + pb * s0)));
        return;
    }
    const int ch = threadIdx.x % FIN_CH, rg = threadIdx.x / FIN_CH;
    const int c = blockIdx.x * FIN_CH + ch;
    double v[4] = {0., 0., 0., 0.};
    if (c < C)
        for (int b = rg; b < blocks; b += FIN_RG) {
            const float *row = p.part + (size_t)b * 4 * C + c;
            double g = 1.0;
            if (split && p.gate)
                g = to_float<TB>(load_bits<TB>((const char *)p.gate + ((size_t)(b / per) * C + c) * TB::SIZE));
            if (p.f) {
                v[0] += g * row[0];
                v[1] += g * row[C];
            }
            if (p.pre != CBR_NORM_NONE) {
                v[2] += row[2 * (size_t)C];
                v[3] += row[3 * (size_t)C];
            }
        }
#pragma unroll
    for (int q = 0; q < 4; ++q) red[q][rg][ch] = v[q];
    for (int half = FIN_RG / 2; half > 0; half /= 2) {
        __syncthreads();
        if (rg < half)
#pragma unroll
            for (int q = 0; q < 4; ++q) red[q][rg][ch] += red[q][rg + half][ch];
    }
    if (rg != 0 || c >= C) return;
    const double s1 = red[0][0][ch], s0 = red[1][0][ch];
    const double w = p.post_w ? p.post_w[c] : 1.0, pb = p.post_b ? p.post_b[c] : 0.0;
    const double r = p.res_scale ? p.res_scale[c] : 1.0, al = p.alpha;
    if (p.dres_scale) p.dres_scale[c] = (float)(al * (w * s1 + pb * s0));
    if (p.dpost_w) p.dpost_w[c] = (float)(al * r * s1);
    if (p.dpost_b) p.dpost_b[c] = (float)(al * r * s0);
    if (p.dpre_w) p.dpre_w[c] = (float)red[2][0][ch];
    if (p.dpre_b) p.dpre_b[c] = (float)red[3][0][ch];
}

using Kernel = void (*)(BlockNormArgs, int, int, int, int);

template <typename TS, typename TB, int E>
Kernel kernel_of(bool tail, bool split)
{
    return tail ? (split ? block_norm_bwd_kernel<TS, TB, E, true, true> : block_norm_bwd_kernel<TS, TB, E, true, false>)
               : (split ? block_norm_bwd_kernel<TS, TB, E, false, true> : block_norm_bwd_kernel<TS, TB, E, false, false>);
}

template <typename TS, typename TB>
hipError_t launch_types(BlockNormArgs a, hipStream_t st)
{
    const Layout o = layout_of(a.C, BWD_THREADS, BWD_THREADS);
    const Deal d = deal_of(a.rows, a.rpg, a.gate != nullptr, o);
    if (!a.gate) a.rpg = a.rows;
    const bool params = a.dres_scale || a.dpost_w || a.dpost_b || a.dpre_w || a.dpre_b;
    const bool gates = a.dgate && d.split;
    if (!params && !gates) a.part = nullptr;
    auto k = o.E == 8 ? kernel_of<TS, TB, 8>(o.tail, d.split) : kernel_of<TS, TB, 16>(o.tail, d.split);
    hipError_t e = launch(k, dim3(d.blocks), dim3(o.threads), 0, st, nullptr, nullptr, a, o.L, o.rpb, d.per, d.gates);
    if (e != hipSuccess || !a.part) return e;
    const int nparam = params ? (a.C + FIN_CH - 1) / FIN_CH : 0;
    const int ngate = gates ? d.blocks / d.per * ((a.C + 255) / 256) : 0;
    return launch(block_norm_bwd_finish_kernel<TB>, dim3(nparam + ngate), dim3(FIN_THREADS), 0, st, nullptr, nullptr, a,
                  d.blocks, d.per, (int)d.split, nparam);
}

}  // namespace

size_t block_norm_part_bytes(uint32_t rows, uint32_t rpg, int C)
{
    const Layout o = layout_of(C, BWD_THREADS, BWD_THREADS);
    int blocks = deal_of(rows, rows, false, o).blocks;
    if (rpg) blocks = std::max(blocks, deal_of(rows, rpg, true, o).blocks);
    return (size_t)blocks * 4 * C * sizeof(float);
}

hipError_t launch_block_norm_bwd(const BlockNormArgs &a, int stream_type, int branch_type, hipStream_t st)
{
    if (stream_type == CBR_BF16) return launch_types<Bf16, Bf16>(a, st);
    if (stream_type == CBR_F16) return launch_types<F16, F16>(a, st);
    if (branch_type == CBR_BF16) return launch_types<F32, Bf16>(a, st);
    if (branch_type == CBR_F16) return launch_types<F32, F16>(a, st);
    return launch_types<F32, F32>(a, st);
}

}  // namespace cbr
