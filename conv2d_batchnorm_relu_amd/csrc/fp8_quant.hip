// fp8_quant.hip -- bf16, f16 or f32 tensors in 8-bit floating point with one scale for each
// group of 128 values of a row, or each 128 x 128 block, of the tensor or of its transpose.
//
//   a = max(largest |v|, fmax 2^-126),  scale = a / fmax,  q = rne(v fmax / a)
// The quotient is the correctly rounded one: with a = m 2^e (m in [1/2, 1)), n = v (fmax 2^-e)
// (fmax is 7 times a power of two: exact for 16-bit sources; of an fp32 one the error is carried
// along), q0 = n (1/m), and one step of Markstein's division, q0 + (n - q0 m)(1/m).  A value midway
// between two 8-bit ones (3/4 of a power of two times the largest, say) is then met exactly and goes
// to the even one; a product with a rounded reciprocal sends a part of them astray.  Quotients of
// 16-bit values that are not midway are 2^-16 of their size off, so fp32 tells them apart; those of
// fp32 values may be 2^-28 off.  There the quotient is rounded to odd: an inexact one has its last
// bit set (one step towards the exact value where it was not), and the rounding to 8 bits goes the
// way that the exact value says.  That is three times the arithmetic, so it is done only where n (1/m)
// moved by 2^-21 of itself up and down rounds to two values: 1 of 2^16 where mantissas are random.
// Bound by memory: 2 or 4 bytes read and 1 written for each value (50176 x 1024 bf16 turned
// over: 28 us = 5.5 TB/s; 64 x 2048: 2.8 us).
#include <type_traits>

#include "block_launch.h"
#include "block_types.h"

namespace cbr {
namespace {

// What turns a group's values into 8 bits: t = v fmax / a (Markstein's correction), then rounding.
template <typename T, bool E5M2>
struct Group {
    float c, m, rm, scale;

    __device__ __forceinline__ void set(float amax)
    {
        constexpr float FMAX = E5M2 ? 57344.f : 448.f;
        const float a = fmaxf(amax, FMAX * 0x1p-126f);
        scale = a / FMAX;
        if (a < __builtin_inff()) {
            const int e = __builtin_amdgcn_frexp_expf(a);
            m = __builtin_amdgcn_frexp_mantf(a);
            c = ldexpf(0.875f, (E5M2 ? 16 : 9) - e);
            rm = 1.f / m;
        } else {   // the finite values of the group become 0, the others NaN
            c = 0.f;
            m = rm = 1.f;
        }
    }
    __device__ __forceinline__ float near(float v) const { return v * c * rm; }   // within 2^-22 of itself
    __device__ __forceinline__ float exact(float v) const
    {
        const float n = v * c, q0 = n * rm;
        if constexpr (T::SIZE == 2) {
            return fmaf(fmaf(-q0, m, n), rm, q0);
        } else {
            const float lo = fmaf(v, c, -n);                                 // n + lo = v c
            const float t = fmaf(fmaf(-q0, m, n) + lo, rm, q0);
            const float r = fmaf(-t, m, n) + lo;                             // (v c / m - t) m
            const int b = __float_as_int(t);
            const bool odd = (b & 1) || !(fabsf(r) > 0.f);                   // odd, exact or NaN: as it is
            return odd ? t : __int_as_float(b + ((b ^ __float_as_int(r)) < 0 ? -1 : 1));
        }
    }
};

// Four values in 8 bits, in order.
template <bool E5M2>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d)
{
    int r = 0;
    if constexpr (E5M2) {
        r = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, r, false);
        r = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, r, true);
    } else {
        r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
        r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
    }
    return (uint32_t)r;
}

// Four values of a group.
template <typename T, bool E5M2>
__device__ __forceinline__ uint32_t encode4(const Group<T, E5M2> &g, float a, float b, float c, float d)
{
    if constexpr (T::SIZE == 4) {
        constexpr float UP = 1.f + 0x1p-21f, DOWN = 1.f - 0x1p-21f;
        const float na = g.near(a), nb = g.near(b), nc = g.near(c), nd = g.near(d);
        const uint32_t up = pack4<E5M2>(na * UP, nb * UP, nc * UP, nd * UP);
        if (__builtin_expect(up == pack4<E5M2>(na * DOWN, nb * DOWN, nc * DOWN, nd * DOWN), 1)) return up;
    }
    return pack4<E5M2>(g.exact(a), g.exact(b), g.exact(c), g.exact(d));
}

// The larger of m and |v|; m where v is a NaN.  The hardware's maximum is one of its operands where
// the other is a quiet NaN, but a NaN where it is a signalling one: those are made quiet first (f16
// ones are when they become float).
template <typename T>
__device__ __forceinline__ float larger(float m, float v)
{
    if constexpr (std::is_same_v<T, F16>) return fmaxf(m, fabsf(v));
    else return fmaxf(m, __builtin_canonicalizef(fabsf(v)));
}

// Eight values of a row at column col, zeros past its end.  The last, partial chunk of a row
// is loaded as the row's last eight values and moved to the front by settle8, once all loads
// are out: value by value, each would be waited for.
template <typename T, bool TAIL>
__device__ __forceinline__ void load8(const char *row, int64_t col, int64_t cols, bool on, Raw8<T> &r)
{
    if (!on || col >= cols) r = Raw8<T>{};
    else if (TAIL && cols < 8) load_part8<T>(row, (int)cols, r);
    else load_raw8<T, TAIL>(row + (TAIL ? min(col, cols - 8) : col) * T::SIZE, r);
}
template <typename T, bool TAIL>
__device__ __forceinline__ void settle8(int64_t col, int64_t cols, Raw8<T> &r)
{
    if (TAIL && cols >= 8) drop8<T>(r, 8 - (int)(cols & 7), col < cols && col + 8 > cols);
}

// Groups of 128 values of a row: sixteen lanes a group, eight values each.  A workgroup takes
// one column of groups over 16 U rows, so the scales of a k block (stored row after row) leave
// as runs of 16 U floats.
constexpr int NT = 256;

template <typename T, bool E5M2, bool TAIL, int U>
__global__ __launch_bounds__(NT) void quant_rows_kernel(const char *__restrict__ src, int64_t rows, int64_t cols,
                                                        int64_t ldq, int kbs, uint8_t *__restrict__ q,
                                                        float *__restrict__ scale)
{
    const int64_t kb = blockIdx.x % kbs, row0 = (int64_t)(blockIdx.x / kbs) * (16 * U);
    const int lane = threadIdx.x % 16, sub = threadIdx.x / 16;
    const int64_t col = kb * 128 + lane * 8;
    Raw8<T> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t row = row0 + u * 16 + sub;
        load8<T, TAIL>(src + row * cols * T::SIZE, col, cols, row < rows, raw[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t row = row0 + u * 16 + sub;
        float v[8], amax = 0.f;
        settle8<T, TAIL>(col, cols, raw[u]);
        unpack8<T>(raw[u], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = larger<T>(amax, v[e]);
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) amax = fmaxf(amax, __shfl_xor(amax, off));
        Group<T, E5M2> g;
        g.set(amax);
        const uint32_t lo = encode4(g, v[0], v[1], v[2], v[3]), hi = encode4(g, v[4], v[5], v[6], v[7]);
        if (row >= rows) continue;
        if (lane == 0) scale[kb * rows + row] = g.scale;
        uint8_t *p = q + row * ldq + col;
        if (col + (TAIL ? 8 : 1) <= cols) {
            *(uint2 *)p = make_uint2(lo, hi);   // ldq and col are multiples of 8
        } else if (TAIL && col < cols) {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < cols - col) p[e] = (uint8_t)((e < 4 ? lo : hi) >> (8 * (e % 4)));
        }
    }
}

// A tile of 128 x 128 source values: the transposed form (groups of 128 down a column), and
// the 128 x 128 blocks of either.  Thread (cl, rl) of 16 x 16 holds rows 8 rl .. + 7 of columns
// 8 cl .. + 7.  The transposed tile is turned over in LDS, 128 bytes of a column padded to 132:
// the 4-byte writes of 16 column groups then fall on different banks but for two at a time.
constexpr int TS = 128, LROW = TS / 4 + 1;

template <typename T, bool E5M2, bool TAIL, bool TRANS, int BLOCK>
__global__ __launch_bounds__(NT) void quant_tile_kernel(const char *__restrict__ src, int64_t rows, int64_t cols,
                                                        int64_t ldq, int ctiles, uint8_t *__restrict__ q,
                                                        float *__restrict__ scale)
{
    __shared__ float red[4][BLOCK == 1 ? TS : 1];
    __shared__ uint32_t turn[TRANS ? TS * LROW : 1];
    __shared__ f32x4 groups[BLOCK == 1 ? TS : 1];
    const int64_t ct = blockIdx.x % ctiles, rt = blockIdx.x / ctiles;
    const int cl = threadIdx.x % 16, rl = threadIdx.x / 16, wave = threadIdx.x / 64;
    const int64_t row0 = rt * TS + rl * 8, col = ct * TS + cl * 8;
    Raw8<T> raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        load8<T, TAIL>(src + (row0 + i) * cols * T::SIZE, col, cols, row0 + i < rows, raw[i]);
    float amax[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) amax[e] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v[8];
        settle8<T, TAIL>(col, cols, raw[i]);
        unpack8<T>(raw[i], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax[e] = larger<T>(amax[e], v[e]);
    }
    Group<T, E5M2> g[BLOCK == 1 ? 8 : 1];
    if constexpr (BLOCK == 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            amax[e] = fmaxf(amax[e], __shfl_xor(amax[e], 16));
            amax[e] = fmaxf(amax[e], __shfl_xor(amax[e], 32));
        }
        if (threadIdx.x % 64 < 16)
#pragma unroll
            for (int e = 0; e < 8; ++e) red[wave][cl * 8 + e] = amax[e];
        __syncthreads();
        // a thread a column works out its group (two divisions: eight columns in every thread
        // took 3 us of the smallest call's 8)
        if (threadIdx.x < TS) {
            const int c = threadIdx.x;
            Group<T, E5M2> w;
            w.set(fmaxf(fmaxf(red[0][c], red[1][c]), fmaxf(red[2][c], red[3][c])));
            groups[c] = f32x4{w.c, w.m, w.rm, w.scale};
            if (ct * TS + c < cols) scale[rt * cols + ct * TS + c] = w.scale;
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const f32x4 w = groups[cl * 8 + e];
            g[e].c = w[0];
            g[e].m = w[1];
            g[e].rm = w[2];
        }
    } else {
        float m = amax[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) m = fmaxf(m, amax[e]);
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) m = fmaxf(m, __shfl_xor(m, off));
        if (threadIdx.x % 64 == 0) red[wave][0] = m;
        __syncthreads();
        g[0].set(fmaxf(fmaxf(red[0][0], red[1][0]), fmaxf(red[2][0], red[3][0])));
        if (threadIdx.x == 0) scale[TRANS ? rt * ctiles + ct : ct * ((rows + TS - 1) / TS) + rt] = g[0].scale;
    }
    if constexpr (!TRANS) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (row0 + i >= rows) break;
            float v[8];
            unpack8<T>(raw[i], v);
            const uint32_t lo = encode4(g[0], v[0], v[1], v[2], v[3]), hi = encode4(g[0], v[4], v[5], v[6], v[7]);
            uint8_t *p = q + (row0 + i) * ldq + col;
            if (col + (TAIL ? 8 : 1) <= cols) {
                *(uint2 *)p = make_uint2(lo, hi);
            } else if (TAIL && col < cols) {
#pragma unroll
                for (int e = 0; e < 7; ++e)
                    if (e < cols - col) p[e] = (uint8_t)((e < 4 ? lo : hi) >> (8 * (e % 4)));
            }
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {   // four rows make a word of each column
            float v[4][8];
#pragma unroll
            for (int i = 0; i < 4; ++i) unpack8<T>(raw[4 * h + i], v[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                turn[(cl * 8 + e) * LROW + rl * 2 + h] = encode4(g[BLOCK == 1 ? e : 0], v[0][e], v[1][e], v[2][e], v[3][e]);
        }
        __syncthreads();
        // eight threads a column, 16 bytes each
#pragma unroll
        for (int pass = 0; pass < TS / 32; ++pass) {
            const int c = pass * 32 + threadIdx.x / 8, k = threadIdx.x % 8 * 16;
            const int64_t out = ct * TS + c, at = rt * TS + k;
            if (out >= cols || at >= rows) continue;
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = turn[c * LROW + k / 4 + i];
            uint8_t *p = q + out * ldq + at;
            if (at + 16 <= rows) {
                *(u32x4 *)p = w;   // ldq and at are multiples of 16
            } else {
                for (int e = 0; e < rows - at; ++e) p[e] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
            }
        }
    }
}

template <typename T, bool E5M2, bool TAIL>
hipError_t launch_form(const cbr_quant_shape &s, const char *src, uint8_t *q, float *scale, hipStream_t st)
{
    const int64_t kbs = (s.cols + 127) / 128, rts = (s.rows + 127) / 128;
    if (s.block == 1 && !s.transpose) {
        // Four rows a thread once that still leaves a workgroup for every CU
        const bool four = rts * 2 * kbs >= 512;
        const int64_t tiles = (s.rows + (four ? 63 : 15)) / (four ? 64 : 16);
        auto k = four ? quant_rows_kernel<T, E5M2, TAIL, 4> : quant_rows_kernel<T, E5M2, TAIL, 1>;
        return launch(k, dim3((uint32_t)(tiles * kbs)), dim3(NT), 0, st, nullptr, nullptr, src, s.rows, s.cols, s.ldq,
                      (int)kbs, q, scale);
    }
    auto k = s.block == 1  ? quant_tile_kernel<T, E5M2, TAIL, true, 1>
             : s.transpose ? quant_tile_kernel<T, E5M2, TAIL, true, 128>
                           : quant_tile_kernel<T, E5M2, TAIL, false, 128>;
    return launch(k, dim3((uint32_t)(rts * kbs)), dim3(NT), 0, st, nullptr, nullptr, src, s.rows, s.cols, s.ldq,
                  (int)kbs, q, scale);
}

template <typename T>
hipError_t launch_type(const cbr_quant_shape &s, const char *src, uint8_t *q, float *scale, hipStream_t st)
{
    const bool e5 = s.q_type == CBR_E5M2, tail = s.cols % 8 != 0;
    if (e5) return tail ? launch_form<T, true, true>(s, src, q, scale, st) : launch_form<T, true, false>(s, src, q, scale, st);
    return tail ? launch_form<T, false, true>(s, src, q, scale, st) : launch_form<T, false, false>(s, src, q, scale, st);
}

}  // namespace

hipError_t launch_fp8_quantize(const cbr_quant_shape &s, const void *src, void *q, float *scale, hipStream_t st)
{
    const char *p = (const char *)src;
    if (s.src_type == CBR_BF16) return launch_type<Bf16>(s, p, (uint8_t *)q, scale, st);
    if (s.src_type == CBR_F16) return launch_type<F16>(s, p, (uint8_t *)q, scale, st);
    return launch_type<F32>(s, p, (uint8_t *)q, scale, st);
}

}  // namespace cbr
