// group_norm.h -- device pieces shared by the group norm's kernels: how a part of an image lies in
// the threads, and sums over the groups.
#pragma once

#include "block_norm.h"

namespace cbr {
namespace gnorm {

using namespace bnorm;   // Row, load_vec, the lane sums

// One workgroup takes `ng` neighbouring groups (a chunk: w = ng * cpg channels, fewer in the last
// one) of `ipw` images, or of one tile of one image's pixels.  Thread (sub, prow, vec) holds the
// chunk's channels 8 vec .. + 7 of image sub, at pixels prow, prow + P, ... : k of them, all in
// registers from the first load to the last store.
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
    float eps;
    Geo g;
};

// Where a workgroup is.  Workgroups go to the eight XCDs in turn, each with its own L2: an XCD takes
// an eighth of them in order, so the chunks that share cache lines of a pixel run beside each other.
// BACK: last first; the second of two kernels begins with what the first one has just read.
template <bool BACK>
struct Place {
    int chunk, tile, c0, w, ngl;   // ngl: groups of this chunk
    int64_t image;                 // the first one
    __device__ __forceinline__ Place(const GroupNormArgs &p, uint32_t total)
    {
        const uint32_t id = blockIdx.x, x = id % 8, q = total / 8, r = total % 8;
        uint32_t t = x * q + min(x, r) + id / 8;
        if (BACK) t = total - 1 - t;
        chunk = t % p.g.chunks;
        t /= p.g.chunks;
        tile = t % p.g.tiles;
        image = (int64_t)(t / p.g.tiles) * p.g.ipw;
        ngl = min(p.g.ng, p.G - chunk * p.g.ng);
        c0 = chunk * p.g.ng * p.cpg;
        w = ngl * p.cpg;
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

// One value of each column (per of them a group, `stride` from an image's first to the next's) summed
// over groups: tot[sub * ng + j].  Short groups by a thread each, longer ones by a (whole) wave.
__device__ __forceinline__ void columns_to_groups(const float *col, float *tot, int per, int stride, int ng, int images)
{
    const int n = images * ng, waves = blockDim.x >> 6;
    if (per <= 8 || waves == 0) {
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            const float *c = col + i / ng * stride + i % ng * per;
            float s = 0.f;
            for (int j = 0; j < per; ++j) s += c[j];
            tot[i] = s;
        }
    } else {
        const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
        if (wave < waves)
            for (int i = wave; i < n; i += waves) {
                const float *c = col + i / ng * stride + i % ng * per;
                float s = 0.f;
                for (int j = lane; j < per; j += 64) s += c[j];
                s = wave_sum(s);
                if (lane == 0) tot[i] = s;
            }
    }
}

// LDS of a workgroup (floats): [rows][NV V ipw] partial sums, [NV V ipw] columns, [ng ipw] groups; `sets` of each.
inline int lds_floats(const Geo &g, int nv, int sets)
{
    const int rows = g.pre ? g.P * g.V / 64 : g.P, wd = nv * g.V * g.ipw;
    return sets * ((rows + 1) * wd + g.ng * g.ipw);
}

// Sums of a group over the pixels and channels that the workgroup holds.  A thread gives NV values: one
// where its eight channels are of one group (cpg % 8 == 0), or eight, one a channel.
template <int NV>
struct GroupSum {
    float *red, *col, *tot;
    int wd, rows, row, at, sub, ng, V;
    bool writes, pre;
    int per;          // columns a group
    __device__ __forceinline__ GroupSum(const GroupNormArgs &p, float *lds, int vec, int prow, int sub_)
    {
        const Geo &g = p.g;
        sub = sub_;
        ng = g.ng;
        V = g.V;
        pre = g.pre;
        wd = NV * V * g.ipw;
        rows = pre ? g.P * V / 64 : g.P;
        row = pre ? prow * V / 64 : prow;
        writes = !pre || (threadIdx.x & 63) < (unsigned)V;
        at = (sub * V + vec) * NV;
        per = NV == 1 ? p.cpg / 8 : p.cpg;
        red = lds;
        col = red + rows * wd;
        tot = col + wd;
    }

    // s: the thread's values; ends with the group's sum for each of them.  gi: group of each.
    __device__ __forceinline__ void operator()(float (&s)[NV], const int (&gi)[NV])
    {
        if (pre) {
            if constexpr (NV == 1) {
                float none[1] = {0.f};
                add_same<1>(s, none, V);
            } else {
                add_same<NV / 2>((float(&)[NV / 2])s[0], (float(&)[NV / 2])s[NV / 2], V);
            }
        }
        if (writes)
#pragma unroll
            for (int e = 0; e < NV; ++e) red[row * wd + at + e] = s[e];
        __syncthreads();
        for (int c = threadIdx.x; c < wd; c += blockDim.x) {
            float v = 0.f;
            for (int r = 0; r < rows; ++r) v += red[r * wd + c];
            col[c] = v;
        }
        __syncthreads();
        columns_to_groups(col, tot, per, NV * V, ng, wd / (NV * V));
        __syncthreads();
#pragma unroll
        for (int e = 0; e < NV; ++e) s[e] = tot[sub * ng + gi[e]];
    }
};

// The group (within the chunk) of each of a thread's values; channels past the chunk: its last group.
template <int NV>
__device__ __forceinline__ void groups_of(int vec, int cpg, int ngl, int (&gi)[NV])
{
    if constexpr (NV == 1) {
        gi[0] = min(8 * vec / cpg, ngl - 1);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) gi[e] = min((8 * vec + e) / cpg, ngl - 1);
    }
}

// exp(-u) by the hardware's exp2 and its reciprocal, both within one last place: sigmoid(u).
__device__ __forceinline__ float sigmoid(float u)
{
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(u * -1.44269504f));
}

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

}  // namespace gnorm
}  // namespace cbr
