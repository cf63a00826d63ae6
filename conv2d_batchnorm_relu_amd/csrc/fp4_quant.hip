// fp4_quant.hip -- bf16, f16 or f32 tensors in 4-bit floating point with an exponent for each group of 32
// values of a row of the tensor or of its transpose, and back.
//
//   a = largest |v|,  scale = 2^(floor(log2 a) - 2),  q = rne(v / scale), at most 6
// The scale is a power of two, so v / scale is exact and the conversion instructions round once; the
// largest value is found on the bits without their sign, whose order is that of the values (NaNs above
// infinity above all numbers).
#include <type_traits>

#include "block_launch.h"
#include "block_types.h"

namespace cbr {
namespace {

constexpr int NT = 256;

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Magnitudes of eight values, as bits: one a word of fp32, two a word of 16-bit types.
template <typename T>
struct Mags {
    uint32_t w[T::WORDS];
    __device__ __forceinline__ void set(const Raw8<T> &r)
    {
        constexpr uint32_t M = T::SIZE == 4 ? 0x7fffffffu : 0x7fff7fffu;
#pragma unroll
        for (int i = 0; i < T::WORDS; ++i) w[i] = r.v[i / 4][i % 4] & M;
    }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b)
    {
        if constexpr (T::SIZE == 4) return max(a, b);
        else
            return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
    }
    __device__ __forceinline__ void join(const Mags &o)
    {
#pragma unroll
        for (int i = 0; i < T::WORDS; ++i) w[i] = larger(w[i], o.w[i]);
    }
    // the largest of the eight, as a value's bits
    __device__ __forceinline__ uint32_t all() const
    {
        uint32_t m = w[0];
#pragma unroll
        for (int i = 1; i < T::WORDS; ++i) m = larger(m, w[i]);
        if constexpr (T::SIZE == 2) m = max(m & 0xffffu, m >> 16);
        return m;
    }
};

// The scale's byte from the largest magnitude's bits: the exponent plus 127, 255 where that is no number.
template <typename T>
__device__ __forceinline__ uint32_t scale_byte(uint32_t mag)
{
    uint32_t e;   // exponent field of the fp32 value
    if constexpr (T::SIZE == 4) e = mag >> 23;
    else if constexpr (std::is_same_v<T, Bf16>) e = mag >> 7;
    else e = __float_as_uint(T::lo(mag)) >> 23;
    return e == 255 ? 255u : (uint32_t)max((int)e - 2, 0);
}

// 2^(byte - 127), also where that is no normal number; the byte is not 255.
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte ? byte << 23 : 0x00400000u); }

// Two values (16-bit types: a word of two) in byte S of `old`.
template <int S>
__device__ __forceinline__ uint32_t pack2(uint32_t old, float a, float b, float scale)
{
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, scale, S);
}
template <typename T, int S>
__device__ __forceinline__ uint32_t pack2(uint32_t old, uint32_t w, float scale)
{
    if constexpr (std::is_same_v<T, Bf16>)
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2, w), scale, S);
    else
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(f16x2, w), scale, S);
}

// Eight values of a group in 32 bits.
template <typename T>
__device__ __forceinline__ uint32_t encode8(const Raw8<T> &r, uint32_t byte)
{
    const float s = scale_of(byte);
    uint32_t q = 0;
    if constexpr (T::SIZE == 4) {
        float v[8];
        unpack8<T>(r, v);
        q = pack2<0>(q, v[0], v[1], s);
        q = pack2<1>(q, v[2], v[3], s);
        q = pack2<2>(q, v[4], v[5], s);
        q = pack2<3>(q, v[6], v[7], s);
    } else {
        q = pack2<T, 0>(q, r.v[0][0], s);
        q = pack2<T, 1>(q, r.v[0][1], s);
        q = pack2<T, 2>(q, r.v[0][2], s);
        q = pack2<T, 3>(q, r.v[0][3], s);
    }
    return byte == 255 ? 0u : q;
}

// Eight values of a row at column col, zeros past its end; a partial last chunk is settled once all loads
// are out (as in the 8-bit quantiser).
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

// Groups of a row: four lanes a group, eight values each; sixteen lanes the four groups of 128 values
// whose scales make a word.  A workgroup takes one column of those over 16 U rows.  (64 x 2048 bf16: 2.7 us, a launch and
// a load.)
template <typename T, bool TAIL, int U>
__global__ __launch_bounds__(NT) void quant4_rows_kernel(const char *__restrict__ src, int64_t rows, int64_t cols, int64_t ldq,
                                                         int kbs, uint8_t *__restrict__ q, uint32_t *__restrict__ scale)
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
    const bool exists = (col & ~31) < cols;   // the lane's group
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t row = row0 + u * 16 + sub;
        settle8<T, TAIL>(col, cols, raw[u]);
        Mags<T> m;
        m.set(raw[u]);
        uint32_t mag = m.all();
        mag = max(mag, (uint32_t)__shfl_xor((int)mag, 1));
        mag = max(mag, (uint32_t)__shfl_xor((int)mag, 2));
        const uint32_t byte = exists ? scale_byte<T>(mag) : 127u, code = encode8<T>(raw[u], byte);
        uint32_t word = byte << (8 * (lane / 4));
        word |= (uint32_t)__shfl_xor((int)word, 4);
        word |= (uint32_t)__shfl_xor((int)word, 8);
        if (row >= rows) continue;
        if (lane == 0) scale[kb * rows + row] = word;
        if (exists) *(uint32_t *)(q + row * ldq + col / 2) = code;
    }
}

// The transpose: a tile of 256 x 64 source values.  Thread (cl, rl) of 8 x 32 holds rows 8 rl .. + 7 of columns
// 8 cl .. + 7; four lanes, eight apart, hold a group of each of their columns.  The codes are turned over in
// LDS: 128 bytes of a column, padded to 132.  Bound by memory: 50176 x 1024 bf16 21 us, 6.1 TB/s (a part of it from the
// caches).
constexpr int TR = 256, TC = 64, LROW = TR / 8 + 1;

template <typename T, bool TAIL>
__global__ __launch_bounds__(NT) void quant4_turned_kernel(const char *__restrict__ src, int64_t rows, int64_t cols, int64_t ldq,
                                                           int ctiles, uint8_t *__restrict__ q, uint8_t *__restrict__ scale)
{
    __shared__ uint32_t turn[TC * LROW];
    __shared__ __attribute__((aligned(16))) uint8_t bytes[2][TC][4];
    const int64_t ct = blockIdx.x % ctiles, rt = blockIdx.x / ctiles;
    const int cl = threadIdx.x % 8, rl = threadIdx.x / 8;
    const int64_t row0 = rt * TR + rl * 8, col = ct * TC + cl * 8;
    Raw8<T> raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) load8<T, TAIL>(src + (row0 + i) * cols * T::SIZE, col, cols, row0 + i < rows, raw[i]);
    Mags<T> m;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        settle8<T, TAIL>(col, cols, raw[i]);
        Mags<T> o;
        o.set(raw[i]);
        if (i == 0) m = o;
        else m.join(o);
    }
#pragma unroll
    for (int i = 0; i < T::WORDS; ++i) {
        m.w[i] = Mags<T>::larger(m.w[i], (uint32_t)__shfl_xor((int)m.w[i], 8));
        m.w[i] = Mags<T>::larger(m.w[i], (uint32_t)__shfl_xor((int)m.w[i], 16));
    }
    const bool exists = (row0 & ~31) < rows;
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) unpack8<T>(raw[i], v[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t mag = T::SIZE == 4 ? m.w[e % T::WORDS] : m.w[e / 2] >> (16 * (e % 2)) & 0xffffu;
        const uint32_t byte = exists ? scale_byte<T>(mag) : 127u;
        const float s = scale_of(byte);
        uint32_t c = 0;
        c = pack2<0>(c, v[0][e], v[1][e], s);
        c = pack2<1>(c, v[2][e], v[3][e], s);
        c = pack2<2>(c, v[4][e], v[5][e], s);
        c = pack2<3>(c, v[6][e], v[7][e], s);
        turn[(cl * 8 + e) * LROW + rl] = byte == 255 ? 0u : c;
        if (rl % 4 == 0) bytes[rl / 16][cl * 8 + e][rl / 4 % 4] = (uint8_t)byte;
    }
    __syncthreads();
    if (threadIdx.x < 2 * TC) {
        const int h = threadIdx.x / TC, c = threadIdx.x % TC;
        const int64_t kb = rt * 2 + h, at = ct * TC + c;
        if (kb * 128 < rows && at < cols) ((uint32_t *)scale)[kb * cols + at] = *(const uint32_t *)bytes[h][c];
    }
    // eight threads a column, 16 bytes (a group) each
#pragma unroll
    for (int pass = 0; pass < TC / 32; ++pass) {
        const int c = pass * 32 + threadIdx.x / 8, k = threadIdx.x % 8;
        const int64_t out = ct * TC + c, at = rt * TR + k * 32;
        if (out >= cols || at >= rows) continue;
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = turn[c * LROW + 4 * k + i];
        *(u32x4 *)(q + out * ldq + at / 2) = w;
    }
}

// Back: eight values a thread.  Bound by memory (50176 x 1024 to bf16: 24 us, 5.4 TB/s; four rows a thread were no faster,
// 4096 x 512 3.8 us instead of 3.2).
template <typename T, bool TAIL>
__global__ __launch_bounds__(NT) void dequant4_kernel(const uint8_t *__restrict__ q, const uint32_t *__restrict__ scale, int64_t rows,
                                                      int64_t cols, int64_t ldq, int kbs, char *__restrict__ v)
{
    const int64_t kb = blockIdx.x % kbs;
    const int lane = threadIdx.x % 16;
    const int64_t row = (int64_t)(blockIdx.x / kbs) * 16 + threadIdx.x / 16, col = kb * 128 + lane * 8;
    if (row >= rows || col >= cols) return;
    const uint32_t code = *(const uint32_t *)(q + row * ldq + col / 2), byte = scale[kb * rows + row] >> (8 * (lane / 4)) & 255u;
    const float s = scale_of(byte);
    float o[8];
    auto two = [&](auto sc) __attribute__((always_inline)) {
        constexpr int S = decltype(sc)::value;
        // unscaled and then multiplied: exact, also for numbers below fp32's normal ones
        const auto p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.f, S);
        o[2 * S] = byte == 255 ? __builtin_nanf("") : p[0] * s;
        o[2 * S + 1] = byte == 255 ? __builtin_nanf("") : p[1] * s;
    };
    two(std::integral_constant<int, 0>{});
    two(std::integral_constant<int, 1>{});
    two(std::integral_constant<int, 2>{});
    two(std::integral_constant<int, 3>{});
    char *p = v + (row * cols + col) * T::SIZE;
    if (!TAIL || col + 8 <= cols) {
        Raw8<T> r;
        pack8<T>(o, r);
        store_raw8<T, TAIL>(p, r);
    } else {
        store_part8<T>(p, (int)(cols - col), o);
    }
}

template <typename T, bool TAIL>
hipError_t launch_quant(const cbr_fp4_shape &s, const char *src, uint8_t *q, uint8_t *scale, hipStream_t st)
{
    if (s.transpose) {
        const int64_t ctiles = (s.cols + TC - 1) / TC, rtiles = (s.rows + TR - 1) / TR;
        return launch(quant4_turned_kernel<T, TAIL>, dim3((uint32_t)(ctiles * rtiles)), dim3(NT), 0, st, nullptr, nullptr, src,
                      s.rows, s.cols, s.ldq, (int)ctiles, q, scale);
    }
    const int64_t kbs = (s.cols + 127) / 128;
    // Four rows a thread where that leaves a CU four workgroups (20000 x 2048 20.0 us, one row 21.3; 4096 x 512, a
    // workgroup a CU, 3.6 and 3.2)
    const bool four = (s.rows + 63) / 64 * kbs >= 1024;
    const int64_t tiles = (s.rows + (four ? 63 : 15)) / (four ? 64 : 16);
    return launch(four ? quant4_rows_kernel<T, TAIL, 4> : quant4_rows_kernel<T, TAIL, 1>, dim3((uint32_t)(tiles * kbs)), dim3(NT), 0,
                  st, nullptr, nullptr, src, s.rows, s.cols, s.ldq, (int)kbs, q, (uint32_t *)scale);
}

template <typename T, bool TAIL>
hipError_t launch_back(const cbr_fp4_shape &s, const uint8_t *q, const uint8_t *scale, char *v, hipStream_t st)
{
    const int64_t rows = s.transpose ? s.cols : s.rows, cols = s.transpose ? s.rows : s.cols, kbs = (cols + 127) / 128;
    return launch(dequant4_kernel<T, TAIL>, dim3((uint32_t)((rows + 15) / 16 * kbs)), dim3(NT), 0, st, nullptr, nullptr, q,
                  (const uint32_t *)scale, rows, cols, s.ldq, (int)kbs, v);
}

}  // namespace

hipError_t launch_fp4_quantize(const cbr_fp4_shape &s, const void *src, void *q, void *scale, hipStream_t st)
{
    const bool tail = s.cols % 8 != 0;
    const char *p = (const char *)src;
    uint8_t *o = (uint8_t *)q, *e = (uint8_t *)scale;
    if (s.type == CBR_BF16) return tail ? launch_quant<Bf16, true>(s, p, o, e, st) : launch_quant<Bf16, false>(s, p, o, e, st);
    if (s.type == CBR_F16) return tail ? launch_quant<F16, true>(s, p, o, e, st) : launch_quant<F16, false>(s, p, o, e, st);
    return tail ? launch_quant<F32, true>(s, p, o, e, st) : launch_quant<F32, false>(s, p, o, e, st);
}

hipError_t launch_fp4_dequantize(const cbr_fp4_shape &s, const void *q, const void *scale, void *v, hipStream_t st)
{
    const bool tail = (s.transpose ? s.rows : s.cols) % 8 != 0;
    const uint8_t *i = (const uint8_t *)q, *e = (const uint8_t *)scale;
    char *o = (char *)v;
    if (s.type == CBR_BF16) return tail ? launch_back<Bf16, true>(s, i, e, o, st) : launch_back<Bf16, false>(s, i, e, o, st);
    if (s.type == CBR_F16) return tail ? launch_back<F16, true>(s, i, e, o, st) : launch_back<F16, false>(s, i, e, o, st);
    return tail ? launch_back<F32, true>(s, i, e, o, st) : launch_back<F32, false>(s, i, e, o, st);
}

}  // namespace cbr
