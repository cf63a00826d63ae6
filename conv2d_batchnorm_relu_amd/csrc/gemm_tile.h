// gemm_tile.h -- device pieces shared by the matrix products of 8- and 4-bit operands: LDS accesses
// and their waits, which tile a workgroup takes, and what happens to a tile's sums.
#pragma once

#include <type_traits>

#include "block_launch.h"
#include "block_types.h"

namespace cbr {
namespace gemm {

typedef __attribute__((address_space(3))) uint8_t lds_u8;

constexpr uint32_t OOB = 0x80000000u;

// The result's side of a product, and how it is divided.
struct TileArgs {
    const float *bias;
    void *d;
    float *part;        // [splits][M][N], where the blocks of k are shared out
    int64_t M;
    int N;
    int d_type, relu;
    int tiles_m, tiles_n, splits;
};

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
struct __attribute__((packed, aligned(2))) Loose8 {
    u32x2 v;
};
struct __attribute__((packed, aligned(4))) LooseF4 {
    f32x4 v;
};

// f(integral_constant 0), ... f(integral_constant N - 1)
template <int N, int I = 0, typename F>
__device__ __forceinline__ void unrolled(F &&f)
{
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        unrolled<N, I + 1>(f);
    }
}

// LDS reads in inline assembly, as in the convolutions: with global-to-LDS loads in flight
// the compiler would wait for all of them before any LDS read of its own.
template <int OFF>
__device__ __forceinline__ u32x4 lds_read16(uint32_t addr)
{
    u32x4 v;
    asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(OFF) : "memory");
    return v;
}
template <int N>
__device__ __forceinline__ void lgkm_wait()
{
    asm volatile("s_waitcnt lgkmcnt(%0)" : : "i"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void vm_wait()
{
    asm volatile("s_waitcnt vmcnt(%0)" : : "i"(N) : "memory");
}
// "At most min(n, MOST) stages of PER loads outstanding."
template <int PER, int MOST>
__device__ __forceinline__ void vm_wait_stages(int n)
{
    if constexpr (MOST == 0) {
        vm_wait<0>();
    } else {
        if (n >= MOST) vm_wait<PER * MOST>();
        else vm_wait_stages<PER, MOST - 1>(n);
    }
}
// Ties a register to the wait before it, so that its use stays behind the wait.
template <typename T>
__device__ __forceinline__ void after_wait(T &x)
{
    asm volatile("" : "+v"(x));
}
template <int OFF>
__device__ __forceinline__ float lds_read4(uint32_t addr)
{
    float v;
    asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(OFF) : "memory");
    return v;
}
// 16 or 4 bytes per lane from buffer offset voff to LDS dst + that times lane (zeros past the end).
__device__ __forceinline__ void buffer_load_lds16(__amdgpu_buffer_rsrc_t r, lds_u8 *dst, int voff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, dst, 16, voff, 0, 0, 0);
}
__device__ __forceinline__ void buffer_load_lds4(__amdgpu_buffer_rsrc_t r, lds_u8 *dst, int voff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, dst, 4, voff, 0, 0, 0);
}

// Four results of consecutive n at (m, n): bias, activation, rounding, store.
__device__ __forceinline__ void finish4(const TileArgs &p, int64_t m, int n, f32x4 v)
{
    const int left = p.N - n;   // > 0
    if (p.bias) {
        if (left >= 4) v += *(const f32x4 *)(p.bias + n);   // n is a multiple of 4
        else
            for (int e = 0; e < 3; ++e)
                if (e < left) v[e] += p.bias[n + e];
    }
    if (p.relu)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = v[e] < 0.f ? 0.f : v[e];   // a NaN stays one
    const int64_t at = m * p.N + n;
    if (p.d_type == CBR_F32) {
        float *o = (float *)p.d + at;
        if (left >= 4) ((LooseF4 *)o)->v = v;
        else
            for (int e = 0; e < 3; ++e)
                if (e < left) o[e] = v[e];
        return;
    }
    const bool half = p.d_type == CBR_F16;
    const uint2 w = half ? make_uint2(F16::pack(v[0], v[1]), F16::pack(v[2], v[3]))
                         : make_uint2(Bf16::pack(v[0], v[1]), Bf16::pack(v[2], v[3]));
    uint16_t *o = (uint16_t *)p.d + at;
    if (left >= 4) ((Loose8 *)o)->v = u32x2{w.x, w.y};
    else
        for (int e = 0; e < 3; ++e)
            if (e < left) o[e] = (uint16_t)((e < 2 ? w.x : w.y) >> (16 * (e & 1)));
}

__device__ __forceinline__ void emit4(const TileArgs &p, int split, int64_t m, int n, f32x4 v)
{
    if (p.part) {
        float *o = p.part + ((int64_t)split * p.M + m) * p.N + n;
        if (n + 4 <= p.N) ((LooseF4 *)o)->v = v;
        else
            for (int e = 0; e < 3; ++e)
                if (n + e < p.N) o[e] = v[e];
    } else {
        finish4(p, m, n, v);
    }
}

// Workgroup -> tile and split.  Workgroups go to the eight XCDs in turn, each with its own L2.
// Where k is shared out, an XCD takes whole splits (all tiles of them: the operands' columns
// of a split are then fetched once) where splits are a multiple of 8.  The plans ask for one, but blocks of k that do not
// divide leave fewer splits, and then two XCDs share some.
// Otherwise it takes an eighth of the tiles, in groups of 8 rows of tiles walked down first,
// so that the tiles that run together share rows of both operands.
__device__ __forceinline__ void place(const TileArgs &p, int &tm, int &tn, int &split)
{
    const uint32_t id = blockIdx.x;
    uint32_t t;
    if (p.splits > 1) {
        split = id % p.splits;
        t = id / p.splits;
    } else {
        const uint32_t all = gridDim.x, x = id % 8, q = all / 8, r = all % 8;
        split = 0;
        t = x * q + min(x, r) + id / 8;
    }
    const uint32_t per = 8u * p.tiles_n, first = t / per * 8, rows = min(8u, p.tiles_m - first);
    t %= per;
    tm = first + t % rows;
    tn = t / rows;
}

// Position of 16-byte chunk c of a row in LDS: c ^ perm.  The sixteen rows that a fragment read
// covers (consecutive ones of a; of b as col_in_wave has them) then fall on all 64 banks.
__device__ constexpr int perm(int row) { return (row >> 1) & 7; }
template <bool F32>
__device__ constexpr int perm_b(int row)
{
    return F32 ? perm(row) : (((row >> 3) & 3) << 1) | ((row >> 1) & 1);
}
// Which of the wave's columns result e of lane group g in product i is (F32: of float outputs,
// four consecutive columns a store).  16-bit outputs: the
// two products of a pair make eight consecutive columns, one 16-byte store, and the four lane
// groups of a row 64 bytes.  (Quads of 8 bytes, 32 bytes a row, made stores the bound:
// 200704 x 128 x 512 took 92 us, 33 without its stores.)
template <bool F32>
__device__ constexpr int col_in_wave(int i, int g, int e)
{
    return F32 ? 16 * i + 4 * g + e : 32 * (i >> 1) + 8 * g + 4 * (i & 1) + e;
}

// A wave's sums: bias, activation, rounding, store.  acc[i][j][e] is the result at row mw + 16 j (a
// lane's own one) and column nl + col_in_wave<F32>(i, 0, e).
template <int MS, int NS, bool F32>
__device__ __forceinline__ void store_tile(const TileArgs &p, const f32x4 (&acc)[NS][MS], int split, int64_t mw, int nl)
{
    // Epilogue: bias (0 without one) and activation (a lower bound: 0, or none), then whole
    // chunks, or value by value in the one that N ends in.
    const bool half = p.d_type == CBR_F16;
    const float *bias = p.part ? nullptr : p.bias;
    const float low = p.relu && !p.part ? 0.f : -__builtin_inff();
    f32x4 bv[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int n = nl + col_in_wave<F32>(i, 0, 0);
        bv[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (bias) {
            if (n + 4 <= p.N) bv[i] = *(const f32x4 *)(bias + n);
            else
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < p.N) bv[i][e] = bias[n + e];
        }
    }
    auto value = [&](int i, int j) __attribute__((always_inline)) {
        f32x4 v = acc[i][j] + bv[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = v[e] < low ? low : v[e];   // a NaN stays one
        return v;
    };
    const int64_t step = 16 * (int64_t)p.N;
    if (F32 || p.part) {
        float *o = (p.part ? p.part + (int64_t)split * p.M * p.N : (float *)p.d) + mw * p.N + nl;
#pragma unroll
        for (int j = 0; j < MS; ++j, o += step)
            if (mw + 16 * j < p.M)
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    const int c = col_in_wave<F32>(i, 0, 0);
                    const f32x4 v = value(i, j);
                    if (nl + c + 4 <= p.N) ((LooseF4 *)(o + c))->v = v;
                    else if (nl + c < p.N)
#pragma unroll
                        for (int e = 0; e < 3; ++e)
                            if (nl + c + e < p.N) o[c + e] = v[e];
                }
    } else {
        uint16_t *o = (uint16_t *)p.d + mw * p.N + nl;
#pragma unroll
        for (int j = 0; j < MS; ++j, o += step)
            if (mw + 16 * j < p.M)
#pragma unroll
                for (int i = 0; i < NS; i += 2) {
                    const int c = col_in_wave<F32>(i, 0, 0);
                    const f32x4 v = value(i, j), w = value(i + 1, j);
                    const u32x4 r = half ? u32x4{F16::pack(v[0], v[1]), F16::pack(v[2], v[3]), F16::pack(w[0], w[1]), F16::pack(w[2], w[3])}
                                         : u32x4{Bf16::pack(v[0], v[1]), Bf16::pack(v[2], v[3]), Bf16::pack(w[0], w[1]), Bf16::pack(w[2], w[3])};
                    if (nl + c + 8 <= p.N) ((Loose16 *)(o + c))->v = r;
                    else if (nl + c < p.N)
#pragma unroll
                        for (int e = 0; e < 7; ++e)
                            if (nl + c + e < p.N) o[c + e] = (uint16_t)(r[e / 2] >> (16 * (e & 1)));
                }
    }
}

// The splits' parts of four results, added in order, and the epilogue (256 threads a workgroup).
__device__ __forceinline__ void join_parts(const TileArgs &p, int splits)
{
    const int q4 = (p.N + 3) / 4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t m = i / q4;
    const int n = (int)(i % q4) * 4;
    if (m >= p.M) return;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    const float *o = p.part + m * p.N + n;
    const int64_t step = p.M * p.N;
    if (n + 4 <= p.N) {
        int s = 0;
        for (; s + 8 <= splits; s += 8) {   // eight loads under way, added in order
            f32x4 w[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) w[u] = ((const LooseF4 *)(o + (s + u) * step))->v;
#pragma unroll
            for (int u = 0; u < 8; ++u) v += w[u];
        }
        for (; s < splits; ++s) v += ((const LooseF4 *)(o + s * step))->v;
    } else {
        for (int s = 0; s < splits; ++s)
            for (int e = 0; e < 3; ++e)
                if (n + e < p.N) v[e] += o[s * step + e];
    }
    finish4(p, m, n, v);
}

}  // namespace gemm
}  // namespace cbr
