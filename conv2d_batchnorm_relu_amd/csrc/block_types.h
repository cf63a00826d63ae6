// block_types.h -- element types of the block norm and the 8-bit kernels: loads and stores
// of eight consecutive values, or of one, in fp32 registers.
#pragma once

#include "cbr_common.h"

namespace cbr {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

struct Bf16 {
    static constexpr int SIZE = 2, WORDS = 4;   // WORDS: 32-bit words of eight values
    static __device__ __forceinline__ float lo(uint32_t v) { return bf16_lo(v); }
    static __device__ __forceinline__ float hi(uint32_t v) { return bf16_hi(v); }
    static __device__ __forceinline__ uint32_t pack(float a, float b) { return pack_bf16x2(a, b); }
};

struct F16 {
    static constexpr int SIZE = 2, WORDS = 4;
    static __device__ __forceinline__ float lo(uint32_t v) { return (float)__builtin_bit_cast(f16x2, v)[0]; }
    static __device__ __forceinline__ float hi(uint32_t v) { return (float)__builtin_bit_cast(f16x2, v)[1]; }
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, f16x2));
    }
};

struct F32 {
    static constexpr int SIZE = 4, WORDS = 8;
};

// Eight values of type T as they sit in memory.
template <typename T>
struct Raw8 {
    u32x4 v[T::WORDS / 4];
};

template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T> &r, float *o)
{
    if constexpr (T::SIZE == 4) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = __uint_as_float(r.v[e / 4][e % 4]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            o[2 * e] = T::lo(r.v[0][e]);
            o[2 * e + 1] = T::hi(r.v[0][e]);
        }
    }
}

template <typename T>
__device__ __forceinline__ void pack8(const float *o, Raw8<T> &r)
{
    if constexpr (T::SIZE == 4) {
#pragma unroll
        for (int e = 0; e < 8; ++e) r.v[e / 4][e % 4] = __float_as_uint(o[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) r.v[0][e] = T::pack(o[2 * e], o[2 * e + 1]);
    }
}

// 16 bytes at an address that is only a multiple of 2: the hardware takes one access for it
// all the same, so rows whose length is no multiple of eight values keep wide accesses.
struct __attribute__((packed, aligned(2))) Loose16 {
    u32x4 v;
};

// Eight values at byte address p: 16-byte aligned, or (LOOSE) at any value's address.
template <typename T, bool LOOSE>
__device__ __forceinline__ void load_raw8(const char *p, Raw8<T> &r)
{
#pragma unroll
    for (int i = 0; i < T::WORDS / 4; ++i)
        if constexpr (LOOSE) r.v[i] = ((const Loose16 *)p)[i].v;
        else r.v[i] = ((const u32x4 *)p)[i];
}

template <typename T, bool LOOSE>
__device__ __forceinline__ void store_raw8(char *p, const Raw8<T> &r)
{
#pragma unroll
    for (int i = 0; i < T::WORDS / 4; ++i)
        if constexpr (LOOSE) ((Loose16 *)p)[i].v = r.v[i];
        else ((u32x4 *)p)[i] = r.v[i];
}

// The bits of the one value at byte address p, in the low part of a word; and back.
template <typename T>
__device__ __forceinline__ uint32_t load_bits(const char *p)
{
    if constexpr (T::SIZE == 4) return *(const uint32_t *)p;
    else return *(const uint16_t *)p;
}

template <typename T>
__device__ __forceinline__ float to_float(uint32_t bits)
{
    if constexpr (T::SIZE == 4) return __uint_as_float(bits);
    else return T::lo(bits);
}

template <typename T>
__device__ __forceinline__ void store_one(char *p, float v)
{
    if constexpr (T::SIZE == 4) *(float *)p = v;
    else *(uint16_t *)p = (uint16_t)T::pack(v, 0.f);
}

// The first n (1..7) of eight values at byte address p; the others read as zero.
template <typename T>
__device__ __forceinline__ void load_part8(const char *p, int n, Raw8<T> &r)
{
    r = Raw8<T>{};
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n) {
            const uint32_t b = load_bits<T>(p + e * T::SIZE);
            if constexpr (T::SIZE == 4) r.v[e / 4][e % 4] = b;
            else r.v[0][e / 2] |= b << (16 * (e % 2));
        }
}

// Moves the last 8 - s of eight values (s = 0..7, the same in all lanes) to the front, zeros
// behind them, in the lanes where `on`.
template <typename T>
__device__ __forceinline__ void drop8(Raw8<T> &r, int s, bool on)
{
    constexpr int W = T::WORDS;
    uint32_t w[W];
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = r.v[i / 4][i % 4];
    auto words = [&](int by) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = on ? (i + by < W ? w[i + by] : 0u) : w[i];
    };
    if (s & 4) words(W / 2);
    if (s & 2) words(W / 4);
    if (s & 1) {
        if constexpr (T::SIZE == 4) words(1);
        else
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = on ? w[i] >> 16 | (i + 1 < W ? w[i + 1] << 16 : 0u) : w[i];
    }
#pragma unroll
    for (int i = 0; i < W; ++i) r.v[i / 4][i % 4] = w[i];
}

template <typename T>
__device__ __forceinline__ void store_part8(char *p, int n, const float *v)
{
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n) store_one<T>(p + e * T::SIZE, v[e]);
}

}  // namespace cbr
