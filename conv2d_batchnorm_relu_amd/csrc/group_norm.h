// group_norm.h -- device pieces shared by the group norm's kernels: how a part of an image lies in
// the threads, and sums over the groups.
#pragma once

#include "block_norm.h"

namespace cbr {
namespace gnorm {

using namespace bnorm;   // Row, load_vec, the lane sums

// One workgroup takes `ng` neighbouring groups (a chunk: w = ng * cpg channels, fewer in the last
// one) of `ipw` images, or of one tile of one image's pixels.  Thread (sub, prow, vec) holds the
// chunk's channels 8 vec .. + 7 of image sub, at pixels prow, prow + P, ...: k of them, all in registers
// from the first load to the last store (a tile's one after the other).
// Pixels a thread holds of an image held whole, of fp32 (twice of 16-bit types): what fits 128 registers with a thread's
// eight channels in one group, in two at most, or each for itself (nv 1, 2, 8).
__host__ __device__ constexpr int fwd_most(int nv) { return nv == 1 ? 10 : nv == 2 ? 8 : 6; }
__host__ __device__ constexpr int bwd_most(int nv) { return nv == 1 ? 4 : nv == 2 ? 3 : 2; }

struct Geo {
    int V, P, ipw;      // vectors of eight channels in a chunk; pixels side by side; images a workgroup
    int ng, chunks;     // groups a chunk, chunks
    int tiles, k;       // tiles of P * k pixels an image
    int pre;            // threads of one image fill whole waves and V divides 64: sums start within the waves
};

struct GroupNormArgs {
    const void *x, *dy;
    void *out;          // y; dx in the backward
    const float *w, *b, *stats_in;
    float *stats, *dw, *db;
    float *part;        // tiles' (mean, M2) of each group; in the backward a tile's two sums of each channel
    int64_t images, pixels;
    int C, G, cpg, act;
    int nt;             // out is written as a stream
    int front;          // workgroups before those of the images (see gn_bwd_apply_kernel)
    float eps;
    Geo g;
};

// Where a workgroup is.  Workgroups go to the eight XCDs in turn, each with its own L2: an XCD takes
// an eighth of them in order, so the chunks that share cache lines of a pixel run beside each other.
struct Place {
    int chunk, tile, c0, w, ngl;   // ngl: groups of this chunk
    int64_t image;                 // the first one
    __device__ __forceinline__ explicit Place(const GroupNormArgs &p)
    {
        const uint32_t id = blockIdx.x - p.front, all = gridDim.x - p.front, x = id % 8, q = all / 8, r = all % 8;
        uint32_t t = x * q + min(x, r) + id / 8;
        chunk = t % p.g.chunks;
        t /= p.g.chunks;
        tile = t % p.g.tiles;
        image = (int64_t)(t / p.g.tiles) * p.g.ipw;
        ngl = min(p.g.ng, p.G - chunk * p.g.ng);
        c0 = chunk * p.g.ng * p.cpg;
        w = ngl * p.cpg;
    }
};

// Where a thread is.
struct Thread {
    int vec, prow, sub, left;   // left: pixels prow, prow + P, ... below it are the thread's
    int64_t image, first;       // its image; the part's first value (of the workgroup's first image)
    bool on;
    __device__ __forceinline__ Thread(const GroupNormArgs &p, const Place &at)
    {
        const Geo &g = p.g;
        const int t = threadIdx.x, q = t / g.V;
        vec = t % g.V;
        prow = q % g.P;
        sub = q / g.P;
        image = at.image + sub;
        const int64_t pixel = (int64_t)at.tile * g.P * g.k;
        const int rows = (int)min((int64_t)g.P * g.k, p.pixels - pixel);
        first = (at.image * p.pixels + pixel) * p.C + at.c0;
        on = image < p.images && 8 * vec < at.w;
        left = on ? rows - prow : 0;
    }
    // how many of the k pixels are the thread's
    __device__ __forceinline__ int pixels(const Geo &g) const { return left > 0 ? min(g.k, (left + g.P - 1) / g.P) : 0; }
};

// A workgroup's part of a tensor: whole chunks of eight channels through a buffer, whose offsets need one
// register for all of a thread's pixels, and without branches: past the end loads read 0 and stores do
// nothing.  (With 64-bit addresses and branches the forward took 40 registers more and held fewer pixels.)
// Every offset formed is below 2^31, those of pixels that are switched off among them (least_time bounds them): what the
// range check makes of a scalar offset past the buffer's end does not matter.
template <typename T, Tail TAIL>
struct Part {
    static constexpr int OOB = (int)0x80000000u;
    char *base;
    __amdgpu_buffer_rsrc_t r;
    int off, step;      // of the thread's first pixel; from one of its pixels to the next (the same for all threads)
    int col, w;         // first channel of the eight, channels of the chunk
    // first: the part's first value; row: the thread's pixel (of C values)
    __device__ __forceinline__ Part(const void *p, int64_t first, int row, int C, int P, int vec, int w_) : col(8 * vec), w(w_)
    {
        base = (char *)p + first * T::SIZE;
        r = __builtin_amdgcn_make_buffer_rsrc(base, 0, 0x7fffffff, 0x00020000);
        off = row * C * T::SIZE;
        step = P * C * T::SIZE;
        if (TAIL == WHOLE) off += col * T::SIZE;
    }
    __device__ __forceinline__ void load(Raw8<T> &o, int i, bool on) const
    {
        if constexpr (TAIL == WHOLE) {
            const int at = on ? off : OOB;
#pragma unroll
            for (int h = 0; h < T::WORDS / 4; ++h)
                o.v[h] = __builtin_amdgcn_raw_buffer_load_b128(r, at + 16 * h, i * step, 0);
        } else {
            const char *row = base + off + (int64_t)i * step;
            if (!on || col >= w) o = Raw8<T>{};
            else if (TAIL == SHORT) load_part8<T>(row, w, o);
            else load_raw8<T, true>(row + (size_t)min(col, w - 8) * T::SIZE, o);
        }
    }
    // The chunk's last, partial eight were loaded as its last eight channels: to the front, zeros behind, once all
    // loads are out.
    __device__ __forceinline__ void settle(Raw8<T> &o) const
    {
        if (TAIL == PART) drop8<T>(o, 8 - (w & 7) & 7, col < w && col + 8 > w);
    }
    // nt: a stream that is not kept in the caches
    __device__ __forceinline__ void store(const float (&v)[8], int i, bool on, bool nt) const
    {
        if constexpr (TAIL == WHOLE) {
            // The offset in one register, none in a scalar one: after a store of 16 bytes with a scalar offset the
            // compiler lets the next instruction write over the data, and lanes 12 to 15 of each 16 stored that.
            const int at = on ? off + i * step : OOB;
            Raw8<T> q;
            pack8<T>(v, q);
            if (nt) {
#pragma unroll
                for (int h = 0; h < T::WORDS / 4; ++h) __builtin_amdgcn_raw_buffer_store_b128(q.v[h], r, at + 16 * h, 0, 2);
            } else {
#pragma unroll
                for (int h = 0; h < T::WORDS / 4; ++h) __builtin_amdgcn_raw_buffer_store_b128(q.v[h], r, at + 16 * h, 0, 0);
            }
        } else if (on) {
            char *q = base + off + (int64_t)i * step + (size_t)col * T::SIZE;
            if (col + 8 <= w) {
                Raw8<T> o;
                pack8<T>(v, o);
                store_raw8<T, true>(q, o);
            } else if (col < w) {
                store_part8<T>(q, w - col, v);
            }
        }
    }
};

// Sum over a whole wave, the same in every lane.
__device__ __forceinline__ float wave_sum(float v)
{
    v = add_across<0>(v);
    v = add_across<1>(v);
    v = add_across<2>(v);
    v = add_across<3>(v);
    v = add_across<4>(v);
    return add_across<5>(v);
}

// How a thread's eight channels fall into groups: all in one (NV 1: cpg % 8 == 0), in two at most (NV 2: cpg > 8; those
// from `bound` on are the second's), or each for itself (NV 8).
template <int NV>
struct Split {
    int gi[NV];     // groups, within the chunk (past the chunk: its last)
    int bound;
    __device__ __forceinline__ Split(int vec, int cpg, int ngl)
    {
        bound = 8;
        if constexpr (NV == 8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) gi[e] = min((8 * vec + e) / cpg, ngl - 1);
        } else {
            const int j = 8 * vec / cpg;
            gi[0] = min(j, ngl - 1);
            if constexpr (NV == 2) {
                gi[1] = min(j + 1, ngl - 1);
                bound = (j + 1) * cpg - 8 * vec;
            }
        }
    }
    __device__ __forceinline__ float pick(const float (&v)[NV], int e) const { return NV == 1 ? v[0] : NV == 8 ? v[NV == 8 ? e : 0] : e < bound ? v[0] : v[NV - 1]; }
    // Values of the eight channels, added up group by group.
    __device__ __forceinline__ void collapse(const float (&c)[8], float (&s)[NV]) const
    {
        if constexpr (NV == 8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = c[e];
        } else {
            float all = 0.f, rest = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (NV == 2) rest += e < bound ? 0.f : c[e];
                all += NV == 2 && e >= bound ? 0.f : c[e];
            }
            s[0] = all;
            s[NV - 1] = NV == 2 ? rest : all;
        }
    }
    // Columns (NV of each vector) that hold group j: from, and how many.  (NV 2: inside a group the second ones are 0.)
    static __host__ __device__ __forceinline__ int from(int j, int cpg)
    {
        return NV == 8 ? j * cpg : NV == 1 ? j * cpg / 8 : 2 * (j * cpg / 8) + (j * cpg % 8 != 0);
    }
    static __host__ __device__ __forceinline__ int count(int j, int cpg)
    {
        return NV == 8 ? cpg : NV == 1 ? cpg / 8 : 2 * (((j + 1) * cpg - 1) / 8) + 1 - from(j, cpg);
    }
};
inline int split_of(int cpg) { return cpg % 8 == 0 ? 1 : cpg > 8 ? 2 : 8; }

// Columns summed over groups: tot[sub * ng + j] of the images' columns, `stride` apart.  Short groups by a thread each,
// longer ones by a (whole) wave.
template <int NV>
__device__ __forceinline__ void columns_to_groups(const float *col, float *tot, int cpg, int stride, int ng, int images)
{
    const int n = images * ng, waves = blockDim.x >> 6;
    if (Split<NV>::count(0, cpg) <= 8 || waves == 0) {
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            const int j = i % ng, m = Split<NV>::count(j, cpg);
            const float *c = col + i / ng * stride + Split<NV>::from(j, cpg);
            float s = 0.f;
            for (int q = 0; q < m; ++q) s += c[q];
            tot[i] = s;
        }
    } else {
        const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
        if (wave < waves)
            for (int i = wave; i < n; i += waves) {
                const int j = i % ng, m = Split<NV>::count(j, cpg);
                const float *c = col + i / ng * stride + Split<NV>::from(j, cpg);
                float s = 0.f;
                for (int q = lane; q < m; q += 64) s += c[q];
                s = wave_sum(s);
                if (lane == 0) tot[i] = s;
            }
    }
}

// Rows of partial sums that the threads of an image leave in LDS: one a wave, or one a pixel lane.
__host__ __device__ inline int sum_rows(const Geo &g) { return g.pre ? g.P * g.V / 64 : g.P; }
// Few enough of them for every thread to add its groups' by itself: one barrier instead of three.
__host__ __device__ inline bool few_rows(const Geo &g, int cpg) { return cpg % 8 == 0 ? sum_rows(g) * (cpg / 8) <= 32 : cpg > 8 && sum_rows(g) * (cpg / 4 + 1) <= 32; }

// Sums of a group over the pixels and channels that the workgroup holds, twice (N values at once).  LDS:
// [2][rows][wd] partial sums, [wd] columns, [ng ipw] groups, wd = NV V ipw, all N times; rounded up to 16 bytes.
__host__ __device__ inline int sum_floats(const Geo &g, int nv, int n) { return (n * ((2 * sum_rows(g) + 1) * nv * g.V * g.ipw + g.ng * g.ipw) + 3) & ~3; }

template <int NV, int N>
struct GroupSum {
    const Geo &g;
    float *red;
    int cpg, wd, rows, row, at, first, turn = 0;
    bool writes, few;
    __device__ __forceinline__ GroupSum(const GroupNormArgs &p, float *lds, const Thread &me) : g(p.g), red(lds), cpg(p.cpg)
    {
        wd = NV * g.V * g.ipw;
        rows = sum_rows(g);
        row = g.pre ? me.prow * g.V / 64 : me.prow;
        writes = !g.pre || (threadIdx.x & 63) < (unsigned)g.V;
        first = me.sub * g.V * NV;
        at = first + me.vec * NV;
        few = NV < 8 && few_rows(g, cpg);
    }

    // s: the thread's values; ends with the group's sum for each of them.
    __device__ __forceinline__ void operator()(float (&s)[N][NV], const Split<NV> &sp)
    {
        if (g.pre) {
            if constexpr (N == 2) add_same<NV>(s[0], s[1], g.V);
            else if constexpr (NV == 1) {
                float none[1] = {0.f};
                add_same<1>(s[0], none, g.V);
            } else {
                add_same<NV / 2>((float(&)[NV / 2])s[0][0], (float(&)[NV / 2])s[0][NV / 2], g.V);
            }
        }
        float *const r0 = red + turn * rows * wd * N;   // [N][rows][wd]
        turn ^= 1;
        if (writes)
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int e = 0; e < NV; ++e) r0[(n * rows + row) * wd + at + e] = s[n][e];
        __syncthreads();
        if (few) {
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                const int m = Split<NV>::count(sp.gi[e], cpg);
                const float *c = r0 + first + Split<NV>::from(sp.gi[e], cpg);
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    float v = 0.f;
                    for (int r = 0; r < rows; ++r)
                        for (int j = 0; j < m; ++j) v += c[(n * rows + r) * wd + j];
                    s[n][e] = v;
                }
            }
            return;
        }
        float *const col = red + 2 * rows * wd * N, *const tot = col + N * wd;
        for (int c = threadIdx.x; c < N * wd; c += blockDim.x) {
            const float *q = r0 + c / wd * rows * wd + c % wd;
            float v = 0.f;
            for (int r = 0; r < rows; ++r) v += q[r * wd];
            col[c] = v;
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) columns_to_groups<NV>(col + n * wd, tot + n * g.ng * g.ipw, cpg, NV * g.V, g.ng, g.ipw);
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < NV; ++e) s[n][e] = tot[n * g.ng * g.ipw + first / (NV * g.V) * g.ng + sp.gi[e]];
    }
};

// SiLU's argument u is held as v = -log2(e) u, so that 2^v = e^-u is one instruction, and
// sigmoid(u) = 1 / (1 + 2^v) comes as -ln 2 sigmoid(u) from a reciprocal of -log2(e) (1 + 2^v): the constants cost
// nothing.  Both hardware functions are within one last place.
constexpr float LOG2E = 1.44269504f, LN2 = 0.693147181f;
// power: 2^v
__device__ __forceinline__ float scaled_sigmoid(float v, float &power)
{
    power = __builtin_amdgcn_exp2f(v);
    return __builtin_amdgcn_rcpf(fmaf(power, -LOG2E, -LOG2E));
}

// LDS of the backward (floats): the groups' sums, and [rows][2][8 V ipw] sums of the channels.
inline int bwd_floats(const Geo &g, int cpg) { return sum_floats(g, split_of(cpg), 2) + 2 * sum_rows(g) * 8 * g.V * g.ipw; }

// How a call is laid out.
Geo plan_group_norm(const cbr_group_norm_shape &s, bool backward);
// Bytes of the parts that workgroups leave for a later kernel (0: none).
inline size_t part_bytes(const cbr_group_norm_shape &s, const Geo &g, bool backward)
{
    const size_t tiles = (size_t)s.images * g.tiles;
    if (backward) return tiles > 1 ? tiles * 2 * s.channels * sizeof(float) : 0;   // one: the sums are the gradients
    return g.tiles > 1 ? tiles * 2 * s.groups * sizeof(float) : 0;
}
// Workgroups of a call, and threads of one.
inline int64_t workgroups(const cbr_group_norm_shape &s, const Geo &g)
{
    return (s.images + g.ipw - 1) / g.ipw * g.tiles * g.chunks;
}
inline int threads_of(const Geo &g) { return g.V * g.P * g.ipw; }
// Outputs past the caches' 32 MB are written as streams: 256 x 28 x 28 x 512
// forward 92 -> 90 us, 8 x 224 x 224 x 64 fp32 backward 113 -> 98, 64 x 56 x 56 x 256 backward 109 -> 95.  With the 4-bit quantiser
// reading the output behind it (and inputs not in the caches), large images gain as much or more (64 x 56 x 56 x 256 backward 128 ->
// 121 us, 8 x 224 x 224 x 64 forward 57 -> 51, bf16), images held whole lose (256 x 28 x 28 x 512 forward 137 -> 146, backward 213 -> 222):
// the 256 MB behind the L2s still hold a part of what they wrote.  Not in runs of fewer than 64 bytes, which the caches
// have to put together (64 x 56 x 56 x 256 backward held whole, in runs of 32: 129 -> 150 us).
inline bool streams(const cbr_group_norm_shape &s, const Geo &g)
{
    const int size = s.type == CBR_F32 ? 4 : 2;
    return s.images * s.pixels * s.channels >= (32 << 20) / size && (int64_t)g.ng * (s.channels / s.groups) * size >= 64;
}

}  // namespace gnorm
}  // namespace cbr
