// fp8_gemm.hip -- matrix product of 8-bit operands with a scale for each block of 128:
//   d[m][n] = act( sum_t sa[t][m] sb[t][n / b_block] * sum_{k in block t} a[m][k] b[n][k] + bias[n] )
//
// A block of 128 is summed by matrix instructions that start from zero; its results are then
// scaled and added to the fp32 sums by the vector unit.  The filter side (b) is the
// instruction's A operand and the activations (a) its B operand, so a lane's four results are
// consecutive n of one m: one scale for all of them when b has 128 x 128 blocks, and one 8- or
// 16-byte store.  Both operands hold k in the same order within a lane, which is all the
// product asks of that order.
//
// Two ways to sum a block:
//   * operands widened to bf16 (exactly) and four v_mfma_f32_16x16x32_bf16, whose sums are
//     fp32 throughout (measured): every call that does not ask for short sums.
//   * v_mfma_f32_16x16x128_f8f6f4, one instruction for the block at twice the rate, for 16-bit
//     outputs of callers that ask for short sums.  It aligns the eight products of each 8
//     consecutive k to the largest of them and keeps 13 bits below its leading one (measured;
//     between eights it adds in fp32).  On normally distributed values that is 1.4e-5 of the
//     result's norm, but products that cancel within an eight take the small ones with them,
//     so it is the caller's choice and never the default.
//     (The few-rows form, bound by reading b, sums in fp32 in any case.)
#include <type_traits>

#include "block_launch.h"
#include "block_types.h"

namespace cbr {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;

constexpr int BK = 128;              // bytes of k in a block, and of an LDS row
constexpr uint32_t OOB = 0x80000000u;

struct GemmArgs {
    const uint8_t *a, *b;
    const float *sa, *sb, *bias;
    void *d;
    float *part;        // [splits][M][N], where the k blocks are shared out
    int64_t M;
    int N, K, lda, ldb;
    int kbs;            // blocks of k
    int kb_per;         // blocks of k a split takes
    int sb_ld;          // scales of b in a block of k
    int d_type, relu;
    int tiles_m, tiles_n, splits;
};

struct __attribute__((packed, aligned(2))) Loose8 {
    uint2 v;
};
struct __attribute__((packed, aligned(4))) LooseF4 {
    f32x4 v;
};

// One product of 16 x 16 over 128 values: FB, FA the formats of b and a (0 e4m3, 1 e5m2).
// Unit scales: the instruction's own (powers of two for 32 values) are not used.
template <int FB, int FA>
__device__ __forceinline__ f32x4 product(const i32x8 &b, const i32x8 &a)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, f32x4{0.f, 0.f, 0.f, 0.f}, FB, FA, 0, 0, 0, 0);
}

// Eight 8-bit values (F: 0 e4m3, 1 e5m2) as bf16, exactly.
template <int F>
__device__ __forceinline__ bf16x8 widen8(uint32_t lo, uint32_t hi)
{
    bf16x2 p[4];
    if constexpr (F == 0) {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
    } else {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.f, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.f, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.f, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.f, true);
    }
    bf16x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = p[e / 2][e % 2];
    return v;
}

// A lane's 32 values of a row of a block, widened: value set t holds bytes 8t..8t+7.
template <int F>
struct Wide {
    bf16x8 t[4];
    __device__ __forceinline__ void set(u32x4 lo, u32x4 hi)
    {
        t[0] = widen8<F>(lo[0], lo[1]);
        t[1] = widen8<F>(lo[2], lo[3]);
        t[2] = widen8<F>(hi[0], hi[1]);
        t[3] = widen8<F>(hi[2], hi[3]);
    }
};

__device__ __forceinline__ f32x4 product(const bf16x8 &b, const bf16x8 &a, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, c, 0, 0, 0);
}

__device__ __forceinline__ i32x8 join(u32x4 lo, u32x4 hi)
{
    return __builtin_bit_cast(i32x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// A sum's two scales as factors x, then y.  A sum q is 0 or within 2^-32 .. 2^39, and q sa sb may
// lie within fp32 where sa sb, or q times one of them, does not.  Scales on the same side of 1 go
// one after the other (each step lies between q and the result), scales on both sides as their
// product (which lies between them).
struct Factors {
    float x, y;
    __device__ __forceinline__ Factors(float sa, float sb)
    {
        const bool same = (fabsf(sa) > 1.f) == (fabsf(sb) > 1.f);
        x = same ? sb : sa * sb;
        y = same ? sa : 1.f;
    }
};
// A sum may always be scaled by a scale within 2^-61 .. 2^60 first, whatever the other one is.
// Whether s lies below or above (0, infinities and NaN: neither).
__device__ __forceinline__ bool tiny(float s) { return __builtin_amdgcn_frexp_expf(s) < -60; }
__device__ __forceinline__ bool huge(float s) { return __builtin_amdgcn_frexp_expf(s) > 60; }

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
__device__ __forceinline__ void finish4(const GemmArgs &p, int64_t m, int n, f32x4 v)
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
    if (left >= 4) ((Loose8 *)o)->v = w;
    else
        for (int e = 0; e < 3; ++e)
            if (e < left) o[e] = (uint16_t)((e < 2 ? w.x : w.y) >> (16 * (e & 1)));
}

__device__ __forceinline__ void emit4(const GemmArgs &p, int split, int64_t m, int n, f32x4 v)
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

// The scales of b for four consecutive n of block kb (BB 1).
__device__ __forceinline__ f32x4 scale4(const GemmArgs &p, int kb, int n)
{
    const float *s = p.sb + (int64_t)kb * p.sb_ld;
    if (n + 4 <= p.N) return ((const LooseF4 *)(s + n))->v;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 3; ++e)
        if (n + e < p.N) v[e] = s[n + e];
    return v;
}

// Workgroup -> tile and split.  Workgroups go to the eight XCDs in turn, each with its own L2.
// Where k is shared out, an XCD takes whole splits (all tiles of them: the operands' columns
// of a split are then fetched once; splits are a multiple of 8 where there are that many).
// Otherwise it takes an eighth of the tiles, in groups of 8 rows of tiles walked down first,
// so that the tiles that run together share rows of both operands.
__device__ __forceinline__ void place(const GemmArgs &p, int &tm, int &tn, int &split)
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

// Tile kernel: 16 MS WM x 16 NS WN results a workgroup, WM x WN waves of 16 MS x 16 NS.
// Both operands' rows of a k block (128 bytes) and their scales come straight into LDS, NST
// blocks deep: while block t is multiplied, blocks t + 1 .. t + NST - 1 are on their way, and
// a wave waits for its own loads of a block by their count, then for the other waves at the
// one barrier a block.  WIDE: through bf16.  F32: float outputs.
// 8192^3, bf16 out: 932 to 966 us = 1.14 to 1.18 PFLOP/s (128 x 128 tiles, four waves), where a
// library's bf16 product takes 901; bound by the matrix unit and by the vector unit that widens and
// scales beside it.  Short sums (256 x 256 tiles): 492 to 496 us = 2.2 PFLOP/s, bound by the
// matrix and vector units taking turns (a block's results are scaled and added by the vector unit:
// 64 instructions to 32 products a wave) and by the barrier of two blocks.
template <int BM, int BN>
constexpr int stage_bytes() { return (BM + BN) * BK + (BM + BN) * 4; }   // rows, then scales

template <int MS, int NS, int WM, int WN, int NST, int FA, int FB, int BB, bool WIDE, bool F32>
__global__ __launch_bounds__(64 * WM * WN, 2) void gemm_tile_kernel(GemmArgs p)
{
    constexpr int NW = WM * WN, BM = 16 * MS * WM, BN = 16 * NS * WN;
    constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;   // load instructions a wave, 8 rows each
    constexpr int PER = LA + LB + 1;                    // and one for the scales
    constexpr int STAGE = stage_bytes<BM, BN>(), SCALES = (BM + BN) * BK;
    static_assert(LA * 8 * NW == BM && LB * 8 * NW == BN && NW >= 2, "tile shape");
    static_assert(32 * NW % BM == 0 && 32 * NW % BN == 0, "half the waves load the scales of a, half those of b");
    static_assert(BB == 1 || 128 % (16 * NS) == 0, "a wave's columns lie in one block of b");
    static_assert(NS % 2 == 0, "products in pairs");
    static_assert(WIDE || !F32, "float outputs have fp32 sums");
    static_assert(MS >= 2, "the next block's loads are issued at the second fragment");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const uint32_t lbase = (uint32_t)(uintptr_t)(lds_u8 *)lds;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    const int wm = wave / WN, wn = wave % WN;

    int tm, tn, split;
    place(p, tm, tn, split);
    const int64_t m0 = (int64_t)tm * BM;
    const int n0 = tn * BN;
    const int kb0 = split * p.kb_per, kb1 = min(p.kbs, kb0 + p.kb_per);

    // rows past the end of an operand lie past the end of its buffer and read as zeros
    const int rows_a = (int)min((int64_t)BM, p.M - m0), rows_b = min(BN, p.N - n0);
    // (256 rows of the longest stride are 2^31 bytes: unsigned)
    const __amdgpu_buffer_rsrc_t ra =
        __builtin_amdgcn_make_buffer_rsrc((void *)(p.a + m0 * p.lda), 0, (int)((uint32_t)rows_a * p.lda), 0x00020000);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc((void *)(p.b + (int64_t)n0 * p.ldb), 0,
                                                                        (int)((uint32_t)rows_b * p.ldb), 0x00020000);
    const int lrow = 8 * wave + (lane >> 3);
    const int lchunk = 16 * ((lane & 7) ^ perm(lrow)), lchunk_b = 16 * ((lane & 7) ^ perm_b<F32>(lrow));
    // 64 scales a wave: of a the first half of the waves, of b the others
    const bool a_scales = wave < NW / 2;
    const int s_at = a_scales ? wave * 64 % BM : (wave - NW / 2) * 64 % BN;
    const int s_lds = SCALES + (a_scales ? s_at : BM + s_at) * 4;
    const int s_len = 4 * (a_scales ? rows_a : BB == 1 ? rows_b : (rows_b + 127) / 128);
    const float *const s_from = a_scales ? p.sa + m0 : p.sb + n0 / BB;
    const int64_t s_ld = a_scales ? p.M : p.sb_ld;
    auto load = [&](int kb, int st) __attribute__((always_inline)) {
        const int kat = kb * BK + lchunk, kbt = kb * BK + lchunk_b;   // a chunk past K is not read: zeros
        lds_u8 *base = (lds_u8 *)lds + st * STAGE;
        lds_u8 *dst = base + wave * 1024;
#pragma unroll
        for (int t = 0; t < LA; ++t)
            buffer_load_lds16(ra, dst + t * NW * 1024, kat < p.K ? (lrow + t * 8 * NW) * p.lda + kat : (int)OOB);
#pragma unroll
        for (int t = 0; t < LB; ++t)
            buffer_load_lds16(rb, dst + BM * BK + t * NW * 1024, kbt < p.K ? (lrow + t * 8 * NW) * p.ldb + kbt : (int)OOB);
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void *)(s_from + kb * s_ld), 0, s_len, 0x00020000);
        buffer_load_lds4(rs, base + s_lds, (s_at + lane) * 4);
    };

    f32x4 acc[NS][MS];
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int j = 0; j < MS; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const uint32_t fa0 = lbase + (wm * 16 * MS + r16) * BK + 16 * (g ^ perm(r16));
    const int brow = col_in_wave<F32>(0, r16 >> 2, r16 & 3);
    const uint32_t fb0 = lbase + (BM + wn * 16 * NS + brow) * BK + 16 * (g ^ perm_b<F32>(brow));
    const uint32_t sa0 = lbase + SCALES + (wm * 16 * MS + r16) * 4;
    const uint32_t sb0 = lbase + SCALES + (BM + wn * 16 * NS + col_in_wave<F32>(0, g, 0)) * 4;   // (BB 1)
    const uint32_t look_a = lbase + SCALES + (wm * 16 * MS + lane % (16 * MS)) * 4;
    const uint32_t look_b = lbase + SCALES + (BM + (BB == 1 ? wn * 16 * NS + lane % (16 * NS) : wn * 16 * NS / 128)) * 4;

    const int turns = kb1 - kb0;
#pragma unroll
    for (int t = 0; t < NST - 1; ++t)
        if (t < turns) load(kb0 + t, t);
    int st = 0;
    for (int t = 0; t < turns; ++t) {
        vm_wait_stages<PER, NST - 2>(turns - 1 - t);
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        const int kb = kb0 + t;
        if (kb + 1 == p.kbs && (p.K & 15)) {
            // the chunk that K ends in: clear what lies past it
            const int kl = p.K - kb * BK, c = kl >> 4, cut = kl & 15;
            for (int r = threadIdx.x; r < BM + BN; r += 64 * NW) {
                u32x4 *q = (u32x4 *)(lds + st * STAGE + r * BK + 16 * (c ^ (r < BM ? perm(r) : perm_b<F32>(r - BM))));
                u32x4 v = *q;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int keep = cut - 4 * e;   // bytes of this word
                    v[e] = keep >= 4 ? v[e] : keep <= 0 ? 0u : v[e] & ((1u << (8 * keep)) - 1u);
                }
                *q = v;
            }
            __syncthreads();
        }
        const uint32_t fa = fa0 + st * STAGE, fb = fb0 + st * STAGE;
        const uint32_t fax = fa ^ 64, fbx = fb ^ 64;
        float s[MS], s1, look[2] = {};
        f32x4 t4[BB == 1 ? NS : 1];
        // The scales of the wave's columns (BB 128: the one), and for BB 128 those of its rows, 64 a
        // read, to see how large they are
        s1 = lds_read4<0>(look_b + st * STAGE);
        if constexpr (BB != 1) {
            look[0] = lds_read4<0>(look_a + st * STAGE);
            if constexpr (MS > 4) look[1] = lds_read4<256>(look_a + st * STAGE);
        }
        u32x4 bf[NS][2], af[3][2];
        auto read = [&]() __attribute__((always_inline)) {
            unrolled<MS>([&](auto jc) __attribute__((always_inline)) {
                constexpr int j = decltype(jc)::value;
                s[j] = lds_read4<j * 64>(sa0 + st * STAGE);
            });
            if constexpr (BB == 1)
                unrolled<NS>([&](auto ic) __attribute__((always_inline)) {
                    constexpr int i = decltype(ic)::value;
                    t4[i] = __builtin_bit_cast(f32x4, lds_read16<col_in_wave<F32>(i, 0, 0) * 4>(sb0 + st * STAGE));
                });
            unrolled<NS>([&](auto ic) __attribute__((always_inline)) {
                constexpr int i = decltype(ic)::value;
                bf[i][0] = lds_read16<col_in_wave<F32>(i, 0, 0) * BK>(fb);
                bf[i][1] = lds_read16<col_in_wave<F32>(i, 0, 0) * BK>(fbx);
            });
            unrolled<2>([&](auto jc) __attribute__((always_inline)) {
                constexpr int j = decltype(jc)::value;
                af[j][0] = lds_read16<j * 16 * BK>(fa);
                af[j][1] = lds_read16<j * 16 * BK>(fax);
            });
        };
        auto wait = [&]() __attribute__((always_inline)) {   // for all of them
            lgkm_wait<0>();
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                after_wait(bf[i][0]);
                after_wait(bf[i][1]);
            }
#pragma unroll
            for (int j = 0; j < MS; ++j) after_wait(s[j]);
            if constexpr (BB == 1)
#pragma unroll
                for (int i = 0; i < NS; ++i) after_wait(t4[i]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                after_wait(af[j][0]);
                after_wait(af[j][1]);
            }
        };
        read();
        // Block t + NST - 1 takes the place of block t - 1: every wave is past its reads (their
        // values went into products) when it reaches the barrier.  Issued among the products:
        // before the block's first reads, the loads held them up by 500 cycles a block (8192^3 with
        // short sums 484 us, 456 right behind the first reads, 454 here).
        auto load_ahead = [&]() __attribute__((always_inline)) {
            if (t + NST - 1 < turns) load(kb + NST - 1, st == 0 ? NST - 1 : st - 1);
        };
        constexpr int AFTER = MS + (BB == 1 ? NS : 0) + 2 * NS + 4;   // reads after the first ones
        lgkm_wait<(AFTER < 15 ? AFTER : 15)>();
        after_wait(s1);
        after_wait(look[0]);
        after_wait(look[1]);
        // Where all are of middling size, each sum is multiplied by the product of its scales (BB 128: one
        // for four results), else by b's and then a's (a multiplication a result more), unless one of
        // b's is tiny and one of a's above 1, or huge and below: see Factors.  A group of zeros has the
        // scale 2^-126, so tiny ones are nothing rare (one row in 16 of each operand: 4096^3 f32 131 ->
        // 151 us; with row-scaled b 136 -> 147, 307 if such blocks went the last way).  Looking costs 2
        // to 5% of a call (8192^3 901 -> 932 us, 1024 x 256 x 50176 40.4 -> 42), 9% with the smallest tiles.
        auto any = [](bool v) __attribute__((always_inline)) { return __builtin_amdgcn_ballot_w64(v) != 0; };
        const bool low = any(tiny(s1)), high = any(huge(s1));
        const bool rows = any(tiny(look[0]) || huge(look[0]) || tiny(look[1]) || huge(look[1]));
        uint32_t how = 0;
        if (__builtin_expect(low || high || rows, 0)) {
            if constexpr (BB == 1) {
                look[0] = lds_read4<0>(look_a + st * STAGE);
                if constexpr (MS > 4) look[1] = lds_read4<256>(look_a + st * STAGE);
                lgkm_wait<0>();
                after_wait(look[0]);
                after_wait(look[1]);
            }
            bool above = false, below = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                above |= fabsf(look[i]) > 1.f;
                below |= look[i] != 0.f && fabsf(look[i]) < 1.f;
            }
            how = (low && any(above)) || (high && any(below)) ? 2 : BB == 1 ? 0 : 1;
        }
        __builtin_amdgcn_sched_barrier(0);
        wait();   // (nothing may be on its way into a register at a branch that does not use it)
        auto multiply = [&](auto by_product) __attribute__((always_inline)) {
            constexpr bool BY_PRODUCT = decltype(by_product)::value;
            if constexpr (BY_PRODUCT)
#pragma unroll
                for (int j = 0; j < MS; ++j) s[j] *= s1;
            f32x4 q[WIDE ? 2 : 1][NS];
            auto add = [&](int i, int j, const f32x4 &v) __attribute__((always_inline)) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[i][j][e] = fmaf(BY_PRODUCT ? v[e] : v[e] * (BB == 1 ? t4[BB == 1 ? i : 0][e] : s1), s[j], acc[i][j][e]);
            };
            if constexpr (WIDE) {
                // Fragment j + 1 is widened, and the products of j - 1 are scaled and added, between
                // the products of j: four vector instructions to a matrix instruction of 16 cycles.
                // (One after the other, both waves of a SIMD did the same at the same time: 2 us more
                // of 1024 x 256 x 50176's 42.)
                Wide<FB> wb[NS];
                Wide<FA> wa[2];
#pragma unroll
                for (int i = 0; i < NS; ++i) wb[i].set(bf[i][0], bf[i][1]);
                wa[0].set(af[0][0], af[0][1]);
                unrolled<MS>([&](auto jc) __attribute__((always_inline)) {
                    constexpr int J = decltype(jc)::value;
                    if constexpr (J + 2 < MS) {   // (its registers were widened two turns ago)
                        af[(J + 2) % 3][0] = lds_read16<(J + 2) * 16 * BK>(fa);
                        af[(J + 2) % 3][1] = lds_read16<(J + 2) * 16 * BK>(fax);
                    }
                    if constexpr (J == MS / 2) load_ahead();
                    if constexpr (J + 1 < MS) {
                        lgkm_wait<(J + 2 < MS ? 2 : 0)>();
                        after_wait(af[(J + 1) % 3][0]);
                        after_wait(af[(J + 1) % 3][1]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int i = 0; i < NS; ++i)
                            q[J % 2][i] = product(wb[i].t[t], wa[J % 2].t[t], t == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : q[J % 2][i]);
                    if constexpr (J + 1 < MS) wa[(J + 1) % 2].set(af[(J + 1) % 3][0], af[(J + 1) % 3][1]);
                    if constexpr (J > 0)
#pragma unroll
                        for (int i = 0; i < NS; ++i) add(i, J - 1, q[(J - 1) % 2][i]);
#pragma unroll
                    for (int u = 0; u < 4 * NS; ++u) {
                        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);   // a matrix instruction
                        __builtin_amdgcn_sched_group_barrier(0x2, 4, 0);   // four of the vector unit
                    }
                    __builtin_amdgcn_sched_barrier(0);
                });
#pragma unroll
                for (int i = 0; i < NS; ++i) add(i, MS - 1, q[(MS - 1) % 2][i]);
            } else {
                unrolled<MS>([&](auto jc) __attribute__((always_inline)) {
                    constexpr int J = decltype(jc)::value;
                    lgkm_wait<(J + 1 < MS ? 2 : 0)>();   // all but the next fragment of a
                    after_wait(af[J % 3][0]);
                    after_wait(af[J % 3][1]);
                    const i32x8 av = join(af[J % 3][0], af[J % 3][1]);
                    if constexpr (J == 1) load_ahead();
#pragma unroll
                    for (int i = 0; i < NS; ++i) {
                        if constexpr (J > 0) add(i, J - 1, q[0][i]);
                        q[0][i] = product<FB, FA>(join(bf[i][0], bf[i][1]), av);
                        // the next fragment but one, once the products that read its registers are under way
                        if constexpr (J + 2 < MS)
                            if (i == 0) {
                                af[(J + 2) % 3][0] = lds_read16<(J + 2) * 16 * BK>(fa);
                                af[(J + 2) % 3][1] = lds_read16<(J + 2) * 16 * BK>(fax);
                            }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                });
#pragma unroll
                for (int i = 0; i < NS; ++i) add(i, MS - 1, q[0][i]);
            }
        };
        // One `if` after another: as two sides of a branch the sums do not stay in place (120 registers spilled).
        if (__builtin_expect(how == 0, 1)) multiply(std::integral_constant<bool, BB != 1>{});
        after_wait(how);
        if constexpr (BB != 1) {
            if (__builtin_expect(__builtin_amdgcn_readfirstlane(how) == 1, 0)) {
                read();
                wait();
                multiply(std::false_type{});
            }
            after_wait(how);
        }
        // Product by product, everything read again, in the order that Factors takes.  Twice the time
        // for such a block.
        if (__builtin_expect(__builtin_amdgcn_readfirstlane(how) == 2, 0)) {
            load_ahead();
            unrolled<MS>([&](auto jc) __attribute__((always_inline)) {
                constexpr int J = decltype(jc)::value;
                u32x4 a0 = lds_read16<J * 16 * BK>(fa), a1 = lds_read16<J * 16 * BK>(fax);
                float sa = lds_read4<J * 64>(sa0 + st * STAGE);
                unrolled<NS>([&](auto ic) __attribute__((always_inline)) {
                    constexpr int I = decltype(ic)::value;
                    u32x4 b0 = lds_read16<col_in_wave<F32>(I, 0, 0) * BK>(fb), b1 = lds_read16<col_in_wave<F32>(I, 0, 0) * BK>(fbx);
                    f32x4 sb;
                    if constexpr (BB == 1)
                        sb = __builtin_bit_cast(f32x4, lds_read16<col_in_wave<F32>(I, 0, 0) * 4>(sb0 + st * STAGE));
                    else
                        sb[0] = s1;
                    lgkm_wait<0>();
                    after_wait(a0);
                    after_wait(a1);
                    after_wait(sa);
                    after_wait(b0);
                    after_wait(b1);
                    after_wait(sb);
                    f32x4 v = {0.f, 0.f, 0.f, 0.f};
                    if constexpr (WIDE) {
                        Wide<FA> wa;
                        Wide<FB> wb;
                        wa.set(a0, a1);
                        wb.set(b0, b1);
#pragma unroll
                        for (int t = 0; t < 4; ++t) v = product(wb.t[t], wa.t[t], v);
                    } else {
                        v = product<FB, FA>(join(b0, b1), join(a0, a1));
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const Factors f(sa, sb[BB == 1 ? e : 0]);
                        acc[I][J][e] = fmaf(v[e] * f.x, f.y, acc[I][J][e]);
                    }
                });
            });
        }
        st = st + 1 == NST ? 0 : st + 1;
    }
    // Epilogue: bias (0 without one) and activation (a lower bound: 0, or none), then whole
    // chunks, or value by value in the one that N ends in.
    const int nl = n0 + wn * 16 * NS + col_in_wave<F32>(0, g, 0);
    const int64_t mw = m0 + wm * 16 * MS + r16;
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

// Few rows of a (m <= 16 MS): bound by reading b once.  A workgroup takes 16 columns, its
// eight waves share the blocks of k, and both operands come from memory straight into the
// product's registers (a row's 128 bytes of a block by four lanes, 64 bytes at a time); the
// waves' sums are added through LDS in wave order.
constexpr int SKW = 8;

template <int MS, int FA, int FB, int BB>
__global__ __launch_bounds__(64 * SKW) void gemm_few_kernel(GemmArgs p)
{
    __shared__ f32x4 red[SKW][MS][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16, nl = n0 + 4 * g;
    const int kb0 = blockIdx.y * p.kb_per, kb1 = min(p.kbs, kb0 + p.kb_per);
    // rows past the end read the last one; their results are not stored
    const uint8_t *brow = p.b + (int64_t)min(n0 + r16, p.N - 1) * p.ldb + 16 * g;
    const uint8_t *arow[MS];
    int mrow[MS];
#pragma unroll
    for (int j = 0; j < MS; ++j) {
        mrow[j] = min(16 * j + r16, (int)p.M - 1);
        arow[j] = p.a + (int64_t)mrow[j] * p.lda + 16 * g;
    }
    f32x4 acc[MS];
#pragma unroll
    for (int j = 0; j < MS; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // One block's operands and scales, as loaded
    struct Block {
        u32x4 b[2], a[MS][2];
        f32x4 sb;
        float sa[MS];
    };
    auto fetch = [&](int kb, Block &o) __attribute__((always_inline)) {
        o.b[0] = *(const u32x4 *)(brow + (int64_t)kb * BK);
        o.b[1] = *(const u32x4 *)(brow + (int64_t)kb * BK + 64);
#pragma unroll
        for (int j = 0; j < MS; ++j) {
            o.a[j][0] = *(const u32x4 *)(arow[j] + (int64_t)kb * BK);
            o.a[j][1] = *(const u32x4 *)(arow[j] + (int64_t)kb * BK + 64);
            o.sa[j] = p.sa[(int64_t)kb * p.M + mrow[j]];
        }
        if constexpr (BB == 1) o.sb = scale4(p, kb, nl);
        else o.sb[0] = p.sb[(int64_t)kb * p.sb_ld + n0 / 128];
    };
    auto multiply = [&](const Block &o) __attribute__((always_inline)) {
        Wide<FB> wb;
        wb.set(o.b[0], o.b[1]);
#pragma unroll
        for (int j = 0; j < MS; ++j) {
            Wide<FA> wa;
            wa.set(o.a[j][0], o.a[j][1]);
            f32x4 q = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 0; t < 4; ++t) q = product(wb.t[t], wa.t[t], q);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const Factors f(o.sa[j], o.sb[BB == 1 ? e : 0]);
                acc[j][e] = fmaf(q[e] * f.x, f.y, acc[j][e]);
            }
        }
    };
    const int full = min(kb1, p.K / BK);   // blocks that K does not end in
    int kb = kb0 + wave;
    if (kb < full) {
        Block now, next;
        fetch(kb, now);
        for (; kb + SKW < full; kb += SKW) {   // the next block loads while this one is multiplied
            fetch(kb + SKW, next);
            multiply(now);
            now = next;
        }
        multiply(now);
    }
    const int last = p.K / BK;
    if (p.K % BK && last >= kb0 && last < kb1 && (last - kb0) % SKW == wave) {
        // the block that K ends in: only 16-byte chunks that begin before K are read, and what
        // lies past K in the last of them is cleared
        const int left = p.K - last * BK - 16 * g;   // bytes from this lane's first chunk on
        auto part = [&](const uint8_t *q, u32x4(&o)[2]) __attribute__((always_inline)) {
            q += (int64_t)last * BK;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                o[h] = left > 64 * h ? *(const u32x4 *)(q + 64 * h) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int keep = left - 64 * h - 4 * e;
                    if (keep < 4) o[h][e] = keep <= 0 ? 0u : o[h][e] & ((1u << (8 * keep)) - 1u);
                }
            }
        };
        Block o;
        part(brow, o.b);
#pragma unroll
        for (int j = 0; j < MS; ++j) {
            part(arow[j], o.a[j]);
            o.sa[j] = p.sa[(int64_t)last * p.M + mrow[j]];
        }
        if constexpr (BB == 1) o.sb = scale4(p, last, nl);
        else o.sb[0] = p.sb[(int64_t)last * p.sb_ld + n0 / 128];
        multiply(o);
    }
#pragma unroll
    for (int j = 0; j < MS; ++j) red[wave][j][lane] = acc[j];
    __syncthreads();
    for (int j = wave; j < MS; j += SKW) {
        f32x4 v = red[0][j][lane];
#pragma unroll
        for (int w = 1; w < SKW; ++w) v += red[w][j][lane];
        const int m = 16 * j + r16;
        if (m < p.M && nl < p.N) emit4(p, blockIdx.y, m, nl, v);
    }
}

// The splits' parts, added in order, and the epilogue.
__global__ __launch_bounds__(256) void gemm_join_kernel(GemmArgs p, int splits)
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

// ------------------------------------------------------------------------------ plan
enum Form { FEW, TILE64, TILE128, TILE256 };

struct GemmPlan {
    Form form;
    int ms;          // FEW: 16-row tiles
    int bm, bn;
    int splits, kb_per;
};

// The tile and the number of splits with the least expected time, in us.  Measured on one
// MI355X: a block of k takes `one` with one workgroup on a CU (256 at a time) and `two` with
// two (512 at a time, the smaller tiles), a workgroup's start and end `ends`, the launch 2.3;
// joining splits takes 4 us and moves each part twice at 4 TB/s.  With short sums the 256-tile
// does twice the arithmetic for each byte that a wave reads from LDS (8192^3: 456 us against 590),
// the 128-tile divides better (12544 x 512 x 2048: 23 us against 38), and a lone workgroup takes
// a block in 0.43 us with a 64-tile, 0.68 with a 128-tile (465 x 1252 x 1540: 9 us against 16;
// 65536 x 64 x 64: 7 against 12); with fp32 sums in 0.67 and 1.0.
struct Costs {
    double one, two, ends;
};

GemmPlan plan_of(const cbr_gemm_shape &s)
{
    const int64_t kbs = (s.k + BK - 1) / BK;
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    GemmPlan best{};
    double least = 0;
    if (s.m <= 64) {
        best.form = FEW;
        best.ms = s.m <= 16 ? 1 : s.m <= 32 ? 2 : 4;
        best.bm = 16 * best.ms;
        best.bn = 16;
        // k shared out among workgroups until every CU has one, two blocks a wave at least
        const int64_t tiles = up(s.n, 16);
        const int64_t splits = tiles < 256 ? std::max<int64_t>(1, std::min(256 / tiles, kbs / (2 * SKW))) : 1;
        best.kb_per = (int)up(kbs, splits);
        best.splits = (int)up(kbs, best.kb_per);
        // b at 6.1 TB/s and, with every 16 columns reading all of a, 3.2% of that for each row
        // (8192 x 8192: 13.1 us for 1 row, 17.8 for 16, 24.7 for 32, 40.2 for 64; tiles take 24)
        least = 2. + (double)s.n * s.k / 6.1e6 * (1. + 0.032 * s.m) + (best.splits > 1 ? 3. : 0.);
    }
    const bool rows = s.b_block == 1, wide = !s.short_sums;   // (short sums: 16-bit outputs only)
    for (const Form form : {TILE64, TILE128, TILE256}) {
        if (form == TILE256 && wide) continue;   // its widened fragments do not fit the registers
        const Costs c = form == TILE256  ? (rows ? Costs{2.15, 0., 6.} : Costs{1.76, 0., 6.})
                        : form == TILE64 ? (wide ? Costs{0.67, 0.9, 2.} : Costs{0.43, 0.52, 1.6})
                        : wide ? (rows ? Costs{1.15, 2.15, 3.} : Costs{1.0, 1.9, 3.})
                                              : (rows ? Costs{0.8, 1.25, 3.} : Costs{0.68, 1.1, 3.});
        const int64_t edge = form == TILE256 ? 256 : form == TILE128 ? 128 : 64, tiles = up(s.m, edge) * up(s.n, edge);
        const int64_t fit = form == TILE256 ? 256 : 512, most = tiles < fit ? std::min(fit / tiles, kbs) : 1;
        for (int64_t want = 1; want <= most; want += want < 8 ? 1 : 8) {   // see place() for eights
            const int64_t per = up(kbs, want), splits = up(kbs, per), wgs = tiles * splits;
            const double t = 2.3 + (wgs <= 256 || form == TILE256 ? up(wgs, 256) * (per * c.one + c.ends)
                                                                  : up(wgs, 512) * (per * c.two + c.ends));
            const double join = splits > 1 ? 4. + (double)splits * s.m * s.n * 8. / 4e6 : 0.;
            if (best.splits == 0 || t + join < least) {
                least = t + join;
                best.form = form;
                best.bm = best.bn = (int)edge;
                best.kb_per = (int)per;
                best.splits = (int)splits;
            }
        }
    }
    return best;
}

template <int MS, int NS, int WM, int WN, int NST, int FA, int FB, int BB, bool WIDE, bool F32>
hipError_t launch_tile(const GemmArgs &a, hipStream_t st)
{
    auto k = gemm_tile_kernel<MS, NS, WM, WN, NST, FA, FB, BB, WIDE, F32>;
    constexpr int lds = NST * stage_bytes<16 * MS * WM, 16 * NS * WN>();
    static_assert(lds <= 160 * 1024, "LDS of a CU");
    const hipError_t e = raise_lds_limit((const void *)k, lds);
    if (e != hipSuccess) return e;
    return launch(k, dim3((uint32_t)a.tiles_m * a.tiles_n * a.splits), dim3(64 * WM * WN), lds, st, nullptr, nullptr, a);
}

template <int FA, int FB, int BB, bool F32>
hipError_t launch_wide(const GemmPlan &pl, bool deep, const GemmArgs &a, hipStream_t st)
{
    if (pl.form == TILE64) return launch_tile<2, 2, 2, 2, 4, FA, FB, BB, true, F32>(a, st);
    return deep ? launch_tile<4, 2, 2, 4, 4, FA, FB, BB, true, F32>(a, st)
                : launch_tile<4, 4, 2, 2, 2, FA, FB, BB, true, F32>(a, st);
}

template <int FA, int FB, int BB>
hipError_t launch_formats(const GemmPlan &pl, bool short_sums, const GemmArgs &a, hipStream_t st)
{
    if (pl.form == FEW) {
        auto k = pl.ms == 1 ? gemm_few_kernel<1, FA, FB, BB>
                 : pl.ms == 2 ? gemm_few_kernel<2, FA, FB, BB> : gemm_few_kernel<4, FA, FB, BB>;
        return launch(k, dim3(a.tiles_n, pl.splits), dim3(64 * SKW), 0, st, nullptr, nullptr, a);
    }
    // one workgroup a CU: four blocks deep; more: two, and two workgroups share a CU
    const bool deep = (int64_t)a.tiles_m * a.tiles_n * pl.splits <= 256;
    if (short_sums) {
        if (pl.form == TILE256) return launch_tile<8, 4, 2, 4, 2, FA, FB, BB, false, false>(a, st);
        if (pl.form == TILE64) return launch_tile<2, 2, 2, 2, 4, FA, FB, BB, false, false>(a, st);
        return deep ? launch_tile<4, 2, 2, 4, 4, FA, FB, BB, false, false>(a, st)
                    : launch_tile<4, 2, 2, 4, 2, FA, FB, BB, false, false>(a, st);
    }
    if (a.d_type == CBR_F32) return launch_wide<FA, FB, BB, true>(pl, deep, a, st);
    return launch_wide<FA, FB, BB, false>(pl, deep, a, st);
}

}  // namespace

size_t gemm_fp8_part_bytes(const cbr_gemm_shape &s)
{
    const GemmPlan p = plan_of(s);
    return p.splits > 1 ? (size_t)p.splits * s.m * s.n * sizeof(float) : 0;
}

hipError_t launch_gemm_fp8(const cbr_gemm_shape &s, const void *a, const float *a_scale, const void *b,
                           const float *b_scale, const float *bias, void *d, float *part, hipStream_t st)
{
    const GemmPlan pl = plan_of(s);
    GemmArgs p{};
    p.a = (const uint8_t *)a;
    p.b = (const uint8_t *)b;
    p.sa = a_scale;
    p.sb = b_scale;
    p.bias = bias;
    p.d = d;
    p.part = pl.splits > 1 ? part : nullptr;
    p.M = s.m;
    p.N = (int)s.n;
    p.K = (int)s.k;
    p.lda = (int)s.lda;
    p.ldb = (int)s.ldb;
    p.kbs = (int)((s.k + BK - 1) / BK);
    p.kb_per = pl.kb_per;
    p.sb_ld = (int)((s.n + s.b_block - 1) / s.b_block);
    p.d_type = s.d_type;
    p.relu = s.relu;
    p.splits = pl.splits;
    p.tiles_m = (int)((s.m + pl.bm - 1) / pl.bm);
    p.tiles_n = (int)((s.n + pl.bn - 1) / pl.bn);
    const bool a5 = s.a_type == CBR_E5M2, b5 = s.b_type == CBR_E5M2, sh = s.short_sums != 0;
    hipError_t e;
    if (s.b_block == 128)
        e = a5 ? (b5 ? launch_formats<1, 1, 128>(pl, sh, p, st) : launch_formats<1, 0, 128>(pl, sh, p, st))
               : (b5 ? launch_formats<0, 1, 128>(pl, sh, p, st) : launch_formats<0, 0, 128>(pl, sh, p, st));
    else
        e = a5 ? (b5 ? launch_formats<1, 1, 1>(pl, sh, p, st) : launch_formats<1, 0, 1>(pl, sh, p, st))
               : (b5 ? launch_formats<0, 1, 1>(pl, sh, p, st) : launch_formats<0, 0, 1>(pl, sh, p, st));
    if (e != hipSuccess || pl.splits == 1) return e;
    const int64_t quads = s.m * ((s.n + 3) / 4);
    return launch(gemm_join_kernel, dim3((uint32_t)((quads + 255) / 256)), dim3(256), 0, st, nullptr, nullptr, p, pl.splits);
}

}  // namespace cbr
