// block_norm.h -- device pieces shared by the block norm's forward and backward kernels:
// how a row's channels lie in the threads, and sums over a row.
#pragma once

#include "block_launch.h"
#include "block_types.h"

namespace cbr {
namespace bnorm {

// A row is held by L threads, E values each (8 or 16): L a power of two up to 64 (then
// several rows share a wave), or a multiple of 64 (several waves share a row).  Thread l's
// values 8i..8i+7 are channels 8 (i L + l) .. + 7, one 16- or 32-byte access.  Tail says what
// the last chunk of a row is: a whole one (C % 8 == 0), a part of one in rows that start at
// any value's address, or (C < 8) a part that is all of the row.
enum Tail { WHOLE = 0, PART = 1, SHORT = 2 };

template <int E>
__device__ __forceinline__ int col_of(int j, int l, int L)
{
    return 8 * ((j >> 3) * L + l) + (j & 7);
}

// Whether value j exists (WHOLE: the same answer for the eight values of a chunk).
template <int E, Tail TAIL>
__device__ __forceinline__ bool has(int j, int l, int L, int C)
{
    return col_of<E>(TAIL ? j : (j & ~7), l, L) < C;
}

// A thread's values of one row of a tensor of type T, as they sit in memory.
template <typename T, int E, Tail TAIL>
struct Row {
    Raw8<T> c[E / 8];

    // row: byte address of the row's channel 0; on false nothing is read and the values are 0.
    // The last, partial chunk of a row is loaded as the row's last eight values and moved to the
    // front when it is used (get): one access like the others, in flight beside the sums.  Value
    // by value, the loads would be waited for here.
    __device__ __forceinline__ void load(const char *row, int l, int L, int C, bool on)
    {
#pragma unroll
        for (int i = 0; i < E / 8; ++i) {
            const int col = 8 * (i * L + l);
            if (!on || col >= C) c[i] = Raw8<T>{};
            else if (TAIL == SHORT) load_part8<T>(row, C, c[i]);
            else load_raw8<T, TAIL == PART>(row + (size_t)(TAIL == PART ? min(col, C - 8) : col) * T::SIZE, c[i]);
        }
    }

    __device__ __forceinline__ void get(float (&o)[E], int l, int L, int C) const
    {
#pragma unroll
        for (int i = 0; i < E / 8; ++i) {
            Raw8<T> r = c[i];
            if (TAIL == PART) {
                const int col = 8 * (i * L + l);
                drop8<T>(r, 8 - (C & 7), col < C && col + 8 > C);
            }
            unpack8<T>(r, o + 8 * i);
        }
    }

    static __device__ __forceinline__ void store(char *row, int l, int L, int C, const float (&v)[E])
    {
#pragma unroll
        for (int i = 0; i < E / 8; ++i) {
            const int col = 8 * (i * L + l);
            char *p = row + (size_t)col * T::SIZE;
            if (col + (TAIL ? 8 : 1) <= C) {
                Raw8<T> r;
                pack8<T>(v + 8 * i, r);
                store_raw8<T, TAIL != WHOLE>(p, r);
            } else if (TAIL && col < C) {
                store_part8<T>(p, C - col, v + 8 * i);
            }
        }
    }
};

// A float vector of the channels, `none` where it is not given.  Through a buffer of its C
// values (none at all without a vector), past whose end loads read 0: no branch, so the loads
// of several vectors are under way together.
template <int E, Tail TAIL>
__device__ __forceinline__ void load_vec(const float *p, float none, int l, int L, int C, float (&o)[E])
{
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void *)p, 0, p ? 4 * C : 0, 0x00020000);
    const float add = p ? 0.f : none;
    if constexpr (TAIL == WHOLE) {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, 4 * col_of<E>(4 * i, l, L), 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[4 * i + e] = __uint_as_float(v[e]) + add;
        }
    } else {   // value by value: no access lies partly past the end
#pragma unroll
        for (int j = 0; j < E; ++j)
            o[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, 4 * col_of<E>(j, l, L), 0, 0)) + add;
    }
}

constexpr int MAX_WAVES = 16;

// v plus the value of the lane across, for the steps of a sum over 2, 4, 8, 16, 32, 64 lanes:
// neighbours, pairs, then quads and eights through mirrored rows (their lanes hold one value
// by then), 16-lane rows and halves by swapping them.  Register moves beside the vector unit:
// a lane shuffle through LDS takes some ten times as long, six of them in a row per sum.
template <int STEP>
__device__ __forceinline__ float add_across(float v)
{
    constexpr int CTRL[4] = {0xB1, 0x4E, 0x141, 0x140};   // quad_perm 1032, 2301; row_half_mirror, row_mirror
    const int b = __float_as_int(v);
    if constexpr (STEP < 4) {
        return v + __int_as_float(__builtin_amdgcn_mov_dpp(b, CTRL[STEP], 0xf, 0xf, true));
    } else {
        // both results hold a row (half) and the one across in the same order at every lane
        const auto r = STEP == 4 ? __builtin_amdgcn_permlane16_swap(b, b, false, false)
                                 : __builtin_amdgcn_permlane32_swap(b, b, false, false);
        return __int_as_float(r[0]) + __int_as_float(r[1]);
    }
}

// One step of the sum over the lanes of a wave that hold the same channels (lane % L): halves
// (STEP 5), 16-lane rows, then rotations within a row (by 8, by 4: the lanes 8 apart hold one
// value by then) and exchanges within quads (1, 0).  Every lane ends with the same sum as those
// it was added to.
template <int STEP>
__device__ __forceinline__ float add_same(float v)
{
    constexpr int ROR = STEP == 3 ? 0x128 : 0x124;   // row_ror:8, row_ror:4
    if constexpr (STEP == 3 || STEP == 2)
        return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), ROR, 0xf, 0xf, true));
    else
        return add_across<STEP>(v);
}

// All steps for the values of two arrays.  One branch a step: with the branches around each
// value (and the code twice) the backward kernel was 16 KB long instead of 8, and a launch of
// few rows waits for its instructions too (196 rows of 256: 13.2 us, 11.3 so).
template <int E, int STEP = 5>
__device__ __forceinline__ void add_same(float (&a)[E], float (&b)[E], int L)
{
    if (L > 1 << STEP) return;
#pragma unroll
    for (int j = 0; j < E; ++j) {
        a[j] = add_same<STEP>(a[j]);
        b[j] = add_same<STEP>(b[j]);
    }
    if constexpr (STEP > 0) add_same<E, STEP - 1>(a, b, L);
}

// Sums over the L threads of each row, for all rows of the workgroup at once: within a wave
// (both operands of an addition are the same at both lanes, so every lane holds the same sum),
// then, for rows of several waves, the waves' sums through LDS in wave order.  Two halves of
// `red` take turns: a wave that is past the barrier of one sum may write the next, never the
// one that others still read.
template <int NV>
struct RowSum {
    float (*red)[MAX_WAVES][NV];   // [2][MAX_WAVES][NV]
    int L, turn;

    template <int STEP>
    __device__ __forceinline__ void step(float (&v)[NV])
    {
        if constexpr (STEP < 6) {
            if (L <= 1 << STEP) return;
#pragma unroll
            for (int e = 0; e < NV; ++e) v[e] = add_across<STEP>(v[e]);
            step<STEP + 1>(v);
        }
    }

    __device__ __forceinline__ void operator()(float (&v)[NV])
    {
        step<0>(v);
        if (L > 64) {
            const int wave = threadIdx.x >> 6, per = L >> 6, first = wave / per * per;
            if ((threadIdx.x & 63) == 0)
#pragma unroll
                for (int e = 0; e < NV; ++e) red[turn][wave][e] = v[e];
            __syncthreads();
#pragma unroll
            for (int e = 0; e < NV; ++e) v[e] = red[turn][first][e];
            for (int i = 1; i < per; ++i)
#pragma unroll
                for (int e = 0; e < NV; ++e) v[e] += red[turn][first + i][e];
            turn ^= 1;
        }
    }
};

// How rows of C channels lie in a workgroup of about `most` threads: eight values a thread
// (one 16-byte access of a 2-byte type) where a row then fits the workgroup, else sixteen.
struct Layout {
    int E, L, rpb, threads;   // values a thread, threads a row, rows a workgroup
    Tail tail;
};

inline Layout layout_of(int C, int most, int limit)
{
    Layout o;
    o.tail = C % 8 == 0 ? WHOLE : C > 8 ? PART : SHORT;
    o.E = (C + 7) / 8 <= limit ? 8 : 16;
    const int n = (C + o.E - 1) / o.E;
    o.L = 1;
    if (n > 64) o.L = (n + 63) / 64 * 64;
    else
        while (o.L < n) o.L *= 2;
    o.rpb = o.L >= most ? 1 : most / o.L;
    o.threads = o.L * o.rpb;
    return o;
}

}  // namespace bnorm
}  // namespace cbr
