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
#include <type_traits>

#include "block_norm.h"

namespace cbr {
namespace {

using namespace bnorm;

// How the rows are dealt out (Deal below).  split: a gate row's rows go to `per` workgroups,
// each within one gate row, and the partial sums are S1, S0, T1, T0 of that gate row.
// Otherwise every group of L threads owns `gates` whole gate rows: it finishes their dgate
// itself and the partial sums are sum g S1, sum g S0, T1, T0.

// Floats from a partial row to the next: four quantities of C channels.
__host__ __device__ constexpr size_t part_ld(int C) { return 4 * (size_t)C; }

constexpr int BWD_THREADS = 512;
// Workgroups that run at once: one of 512 threads a CU (137 to 256 registers a thread).  With
// two or three times as many, or with two on a CU at 128 registers, the partial rows and the
// spilled registers cost more than the waves hide (4096 x 4096, when this was chosen: 78 us; 512
// workgroups 91, at 128 registers 114, 768 of 256 threads 99).
constexpr int BWD_BLOCKS = 256;

struct Deal {
    Layout o;
    int blocks, per, gates;
    bool split;
};

Deal deal_of(uint32_t rows, uint32_t rpg, bool gate, int C)
{
    const uint64_t gates = gate ? rows / rpg : 1;
    if (!gate) rpg = rows;
    auto up = [](uint64_t a, uint64_t b) { return (a + b - 1) / b; };
    Deal d;
    d.o = layout_of(C, BWD_THREADS, BWD_THREADS);
    const uint64_t subs = (uint64_t)BWD_BLOCKS * d.o.rpb;
    // Rows in turn of the busiest group of threads either way; a workgroup's start and end (its
    // coefficients, its partial row) cost about eight.
    const uint64_t per = std::max<uint64_t>(1, std::min<uint64_t>(BWD_BLOCKS / gates, rpg / d.o.rpb));
    const uint64_t split_turns = up(gates * per, BWD_BLOCKS) * (up(up(rpg, per), d.o.rpb) + 8);
    const uint64_t whole_turns = up(gates, subs) * rpg + 8;
    d.split = !gate || split_turns < whole_turns;
    if (d.split) {
        d.per = (int)per;
        d.gates = 1;
        d.blocks = (int)(gates * per);
    } else {
        d.per = 1;
        d.gates = (int)up(gates, subs);
        const uint64_t groups = up(gates, d.gates);
        // few groups: in smaller workgroups, to reach every CU
        if (groups < subs / 2) d.o = layout_of(C, BWD_THREADS / 2, BWD_THREADS);
        d.blocks = (int)up(groups, d.o.rpb);
    }
    return d;
}

// Bound by memory (dy, dh, y, f read once, dx, df written once) where the rows are many, by
// the latency of two sums over a row and of the next row's loads where they are few: 4096 x
// 4096 (f32 stream, bf16 branch) 71 us = 4.3 TB/s, 64 x 56 x 56 x 256 with a gate an image 134 us
// = 4.6 TB/s, of 5.2 that a copy reaches.  Two waves a SIMD are what one workgroup a CU gives: the
// compiler may use all of the registers that leaves, and is told so.
template <typename TS, typename TB, int E, Tail TAIL, bool SPLIT>
__global__ __launch_bounds__(BWD_THREADS) __attribute__((amdgpu_waves_per_eu(2, 2))) void
block_norm_bwd_kernel(BlockNormArgs p, int L, int rpb, int per, int gates)
{
    __shared__ float red[2][MAX_WAVES][2];
    constexpr int COMB = BWD_THREADS * E;
    __shared__ float comb[E > 8 ? 1 : 4 * COMB];   // (sixteen values a thread: a row takes the whole workgroup)
    RowSum<2> sum{red, L, 0};
    const int C = p.C, l = threadIdx.x % L, sub = threadIdx.x / L;
    const bool hasf = p.f != nullptr, haspre = p.pre != CBR_NORM_NONE, haspost = p.post != CBR_NORM_NONE;

    // This thread group's rows: r0 + t * step for t < turns, those below r1 existing.
    uint64_t r0, r1;
    uint32_t step, turns;
    if constexpr (SPLIT) {
        const uint32_t gi = blockIdx.x / per, part = blockIdx.x % per;
        const uint32_t own = p.rpg / per, more = p.rpg % per;   // the first `more` take one more
        const uint64_t a = (uint64_t)gi * p.rpg + part * own + min(part, more);
        const uint32_t mine = own + (part < more);
        r0 = a + sub;
        r1 = a + mine;
        step = rpb;
        turns = (mine + rpb - 1) / rpb;
    } else {
        const uint64_t own = (uint64_t)gates * p.rpg;
        r0 = ((uint64_t)blockIdx.x * rpb + sub) * own;
        r1 = r0 + own < p.rows ? r0 + own : p.rows;
        step = 1;
        turns = (uint32_t)own;
    }

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
    // The first row, the gate and the vectors are asked for together, and a row's loads run
    // beside the sums of the row before it; with sixteen values a thread there are no registers
    // for that (up to 160 spilled), so a row is loaded when its turn comes.
    Row<TB, E, TAIL> graw;
    constexpr bool AHEAD = E == 8;
    if constexpr (AHEAD) fetch(r0);
    if constexpr (SPLIT)
        graw.load((const char *)p.gate + (uint64_t)(blockIdx.x / per) * C * TB::SIZE, l, L, C, p.gate != nullptr);
    // alpha r post_w (SPLIT: times g), pre_w, and for whole gate rows' dgate alpha r post_b (sixteen
    // values a thread: loaded when a gate row ends, there are no registers for them)
    constexpr bool KEEP = !SPLIT && E == 8;
    float cw[E], pw[E], cb[KEEP ? E : 1];
    auto load_cb = [&](float(&o)[E]) __attribute__((always_inline)) {
        float v[E];
        load_vec<E, TAIL>(p.post_b, 0.f, l, L, C, o);
        load_vec<E, TAIL>(p.res_scale, 1.f, l, L, C, v);
#pragma unroll
        for (int j = 0; j < E; ++j) o[j] *= p.alpha * v[j];
    };
    if constexpr (KEEP) load_cb(cb);
    {
        float w[E];
        load_vec<E, TAIL>(p.res_scale, 1.f, l, L, C, cw);
        load_vec<E, TAIL>(p.post_w, 1.f, l, L, C, w);
        load_vec<E, TAIL>(p.pre_w, 1.f, l, L, C, pw);
#pragma unroll
        for (int j = 0; j < E; ++j) cw[j] *= p.alpha * w[j];
        if (SPLIT && p.gate) {
            graw.get(w, l, L, C);
#pragma unroll
            for (int j = 0; j < E; ++j) cw[j] *= w[j];
        }
    }
    float s1[E], s0[E], t1[E], t0[E], g1[E], g0[E];   // (g1, g0: !SPLIT)
#pragma unroll
    for (int j = 0; j < E; ++j) s1[j] = s0[j] = t1[j] = t0[j] = 0.f;
#pragma unroll
    for (int j = 0; j < E; ++j) g1[j] = g0[j] = 0.f;

    uint32_t left = p.rpg;   // rows left of the current gate row (!SPLIT)
    for (uint32_t t = 0; t < turns; ++t) {
        const uint64_t row = r0 + (uint64_t)t * step;
        const bool on = row < r1;
        if constexpr (!AHEAD) fetch(row);
        float d[E], a[E], b[E], f[E];
        dyn.get(d, l, L, C);
        yn.get(a, l, L, C);
        dhn.get(b, l, L, C);
        fn.get(f, l, L, C);
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
                if (p.gate) graw.get(g, l, L, C);
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
                d[j] *= cw[j];
                if constexpr (!SPLIT) d[j] *= g[j];
                if (haspost) {
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
                        float o[E];
#pragma unroll
                        for (int j = 0; j < E; ++j) o[j] = cw[j] * s1[j];
                        if (p.post_b) {
                            float b[E];
                            if constexpr (!KEEP) load_cb(b);
#pragma unroll
                            for (int j = 0; j < E; ++j) o[j] = fmaf(KEEP ? cb[KEEP ? j : 0] : b[j], s0[j], o[j]);
                        }
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
    // The workgroup's partial row: a pair of sums at a time, added over the lanes of a wave that
    // hold the same channels, then over the waves (rows of several waves: over the rows) in order.
    const int slots = L < 64 ? (int)(blockDim.x >> 6) : rpb, slot = L < 64 ? (int)(threadIdx.x >> 6) : sub;
    const int first = hasf ? 0 : 1, pairs = haspre ? 2 : 1;
    float *const out = p.part + blockIdx.x * part_ld(C);
#pragma unroll 1
    for (int pair = first; pair < pairs; ++pair) {   // (a loop: the code once)
        float u1[E], u0[E];
#pragma unroll
        for (int j = 0; j < E; ++j) {
            u1[j] = pair ? t1[j] : SPLIT ? s1[j] : g1[j];
            u0[j] = pair ? t0[j] : SPLIT ? s0[j] : g0[j];
        }
        if (L < 64) add_same<E>(u1, u0, L);
        if (E > 8 || slots == 1) {   // nothing to add
            if (threadIdx.x < (uint32_t)L) {
                Row<F32, E, TAIL>::store((char *)(out + 2 * (size_t)pair * C), l, L, C, u1);
                Row<F32, E, TAIL>::store((char *)(out + (2 * (size_t)pair + 1) * C), l, L, C, u0);
            }
        } else if (L >= 64 || (threadIdx.x & 63) < L) {
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int at = slot * L * E + col_of<E>(j, l, L);
                comb[2 * pair * COMB + at] = u1[j];
                comb[(2 * pair + 1) * COMB + at] = u0[j];
            }
        }
    }
    if (E > 8 || slots == 1) return;
    __syncthreads();
    for (int i = threadIdx.x + 2 * first * C; i < 2 * pairs * C; i += blockDim.x) {
        const int q = (i >= C) + (i >= 2 * C) + (i >= 3 * C);
        const float *from = comb + q * COMB + (i - q * C);
        float v = from[0];
        int s = 1;
        for (; s + 4 <= slots; s += 4) {   // four reads under way, added in order
            const float a = from[s * L * E], b = from[(s + 1) * L * E];
            const float d = from[(s + 2) * L * E], f = from[(s + 3) * L * E];
            v = v + a + b + d + f;
        }
        for (; s < slots; ++s) v += from[s * L * E];
        out[i] = v;
    }
}

// The parameters' gradients from the partial rows, in fp64 and a fixed order.  Blocks
// 0 .. nparam - 1 take 64 channels of one norm's pair of sums each: sixteen waves share the
// partial rows (a wave reads 256 bytes of a row, FIN_UN rows' loads under way together) and
// are added through LDS in wave order.  (Lane shuffles of fp64 values cost more than the
// loads: 6.6 us against 4 on the smallest case.)  The blocks after them (dgate of a split
// gate row): of one gate row, 64 channels shared by the waves in the same way, or 1024 where
// there are few partial rows, a thread a channel.
// The parameter vectors are read through buffers whose length says what exists, so without
// branches and beside the sums' loads.
constexpr int FIN_RG = 16, FIN_THREADS = 64 * FIN_RG, FIN_UN = 8;

// Value c of n floats at p (p NULL or c past the end: `none`).
__device__ __forceinline__ float float_at(const float *p, int n, int c, float none)
{
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void *)p, 0, p ? 4 * n : 0, 0x00020000);
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, 4 * c, 0, 0)) + (p ? 0.f : none);
}
template <typename TB>
__global__ __launch_bounds__(FIN_THREADS) void block_norm_bwd_finish_kernel(BlockNormArgs p, int blocks, int per,
                                                                            int split, int nparam)
{
    __shared__ double red[2][FIN_RG][64];
    const int C = p.C;
    if ((int)blockIdx.x >= nparam) {
        // the gate row's `per` partial rows
        const bool wide = per >= FIN_RG / 2;
        const int width = wide ? 64 : FIN_THREADS, tiles = (C + width - 1) / width, b = blockIdx.x - nparam;
        const int gi = b / tiles, c = b % tiles * width + threadIdx.x % width;
        const int k0 = wide ? __builtin_amdgcn_readfirstlane(threadIdx.x / 64) : 0, step = wide ? FIN_RG : 1;
        const size_t ld = part_ld(C);
        double s1 = 0., s0 = 0.;
        const float w = float_at(p.post_w, C, c, 1.f), pb = float_at(p.post_b, C, c, 0.f);
        const float res = float_at(p.res_scale, C, c, 1.f);
        if (c < C) {
            const float *row = p.part + (size_t)gi * per * ld + c;
            for (int k = k0; k < per; k += 4 * step) {
                float a[4], z[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const size_t at = min(k + u * step, per - 1) * ld;   // past the end: read, not added
                    a[u] = row[at];
                    z[u] = row[at + C];
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (k + u * step < per) {
                        s1 += a[u];
                        s0 += z[u];
                    }
            }
        }
        if (wide) {
            red[0][k0][threadIdx.x % 64] = s1;
            red[1][k0][threadIdx.x % 64] = s0;
            __syncthreads();
            if (k0 != 0) return;
            for (int i = 1; i < FIN_RG; ++i) {
                s1 += red[0][i][threadIdx.x];
                s0 += red[1][i][threadIdx.x];
            }
        }
        if (c >= C) return;
        const double ar = (double)p.alpha * res;
        store_one<TB>((char *)p.dgate + ((size_t)gi * C + c) * TB::SIZE, (float)(ar * ((double)w * s1 + (double)pb * s0)));
        return;
    }
    const bool hasf = p.f != nullptr, haspre = p.pre != CBR_NORM_NONE;
    // which pair: the post norm's S1, S0 or the pre norm's T1, T0 (those that exist)
    const bool post = hasf && (!haspre || blockIdx.x % 2 == 0);
    const int c = (hasf && haspre ? blockIdx.x / 2 : blockIdx.x) * 64 + threadIdx.x % 64;
    const int rg = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);   // the addresses' arithmetic is scalar
    const bool weigh = post && split && p.gate;
    const float w = float_at(p.post_w, C, c, 1.f), pb = float_at(p.post_b, C, c, 0.f);
    const float res = float_at(p.res_scale, C, c, 1.f);
    double s1 = 0., s0 = 0.;
    auto add = [&](auto un) __attribute__((always_inline)) {   // `un` partial rows at a time
        constexpr int UN = decltype(un)::value;
        const float *rows = p.part + (post ? 0 : 2 * (size_t)C) + c;
        for (int b0 = rg; b0 < blocks; b0 += FIN_RG * UN) {
            float a[UN], z[UN];
            uint32_t g[UN];
#pragma unroll
            for (int u = 0; u < UN; ++u) {
                const int b = min(b0 + u * FIN_RG, blocks - 1);   // past the end: read, not added
                a[u] = rows[b * part_ld(C)];
                z[u] = rows[b * part_ld(C) + C];
            }
            if (weigh)
#pragma unroll
                for (int u = 0; u < UN; ++u)
                    g[u] = load_bits<TB>((const char *)p.gate +
                                         ((size_t)(min(b0 + u * FIN_RG, blocks - 1) / per) * C + c) * TB::SIZE);
#pragma unroll
            for (int u = 0; u < UN; ++u)
                if (b0 + u * FIN_RG < blocks) {
                    const double gv = weigh ? to_float<TB>(g[u]) : 1.f;
                    s1 += gv * a[u];
                    s0 += gv * z[u];
                }
        }
    };
    if (c < C) {
        if (blocks > FIN_RG) add(std::integral_constant<int, FIN_UN>{});
        else add(std::integral_constant<int, 1>{});
    }
    red[0][rg][threadIdx.x % 64] = s1;
    red[1][rg][threadIdx.x % 64] = s0;
    __syncthreads();
    if (rg != 0 || c >= C) return;
    for (int i = 1; i < FIN_RG; ++i) {
        s1 += red[0][i][threadIdx.x];
        s0 += red[1][i][threadIdx.x];
    }
    if (post) {
        const double r = res, al = p.alpha;
        if (p.dres_scale) p.dres_scale[c] = (float)(al * ((double)w * s1 + (double)pb * s0));
        if (p.dpost_w) p.dpost_w[c] = (float)(al * r * s1);
        if (p.dpost_b) p.dpost_b[c] = (float)(al * r * s0);
    } else {
        if (p.dpre_w) p.dpre_w[c] = (float)s1;
        if (p.dpre_b) p.dpre_b[c] = (float)s0;
    }
}

using Kernel = void (*)(BlockNormArgs, int, int, int, int);

template <typename TS, typename TB, int E, Tail TAIL>
Kernel kernel_of(bool split)
{
    return split ? block_norm_bwd_kernel<TS, TB, E, TAIL, true> : block_norm_bwd_kernel<TS, TB, E, TAIL, false>;
}

template <typename TS, typename TB>
hipError_t launch_types(BlockNormArgs a, hipStream_t st)
{
    const Deal d = deal_of(a.rows, a.rpg, a.gate != nullptr, a.C);
    const Layout &o = d.o;
    if (!a.gate) a.rpg = a.rows;
    const bool params = a.dres_scale || a.dpost_w || a.dpost_b || a.dpre_w || a.dpre_b;
    const bool gates = a.dgate && d.split;
    if (!params && !gates) a.part = nullptr;
    auto k = o.E == 16 ? (o.tail == WHOLE ? kernel_of<TS, TB, 16, WHOLE>(d.split) : kernel_of<TS, TB, 16, PART>(d.split))
             : o.tail == WHOLE  ? kernel_of<TS, TB, 8, WHOLE>(d.split)
             : o.tail == PART ? kernel_of<TS, TB, 8, PART>(d.split) : kernel_of<TS, TB, 8, SHORT>(d.split);
    hipError_t e = launch(k, dim3(d.blocks), dim3(o.threads), 0, st, nullptr, nullptr, a, o.L, o.rpb, d.per, d.gates);
    if (e != hipSuccess || !a.part) return e;
    const int pairs = (a.f != nullptr) + (a.pre != CBR_NORM_NONE);
    const int nparam = params ? pairs * ((a.C + 63) / 64) : 0;
    const int width = d.per >= FIN_RG / 2 ? 64 : FIN_THREADS;   // channels of a dgate block, as the kernel has it
    const int ngate = gates ? d.blocks / d.per * ((a.C + width - 1) / width) : 0;
    return launch(block_norm_bwd_finish_kernel<TB>, dim3(nparam + ngate), dim3(FIN_THREADS), 0, st, nullptr, nullptr, a,
                  d.blocks, d.per, (int)d.split, nparam);
}

}  // namespace

size_t block_norm_part_bytes(uint32_t rows, uint32_t rpg, int C)
{
    int blocks = deal_of(rows, rows, false, C).blocks;
    if (rpg) blocks = std::max(blocks, deal_of(rows, rpg, true, C).blocks);
    return blocks * part_ld(C) * sizeof(float);
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
