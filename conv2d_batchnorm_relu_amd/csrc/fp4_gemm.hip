// fp4_gemm.hip -- matrix product of 4-bit operands with an exponent for each 32 values of k:
//   d[m][n] = act( sum_t 2^(ea[m][t] + eb[n][t]) sum_{k in group t} a[m][k] b[n][k] + bias[n] )
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes four groups of 32 and their exponents and adds to its fp32
// sums.  Measured: a group's sum is exact (its products have 8 bits between the largest and the last), and sums are while
// fp32 holds them.  Where groups are added whose sizes differ, the smaller keeps its bits down to 2^-23 of a large sum, or to
// 2^-22 of a large product, which is aligned by its largest possible value.  Sums of one sign: 1024 x 256 x 50176 with exponents
// over 2^20 within 6 2^-23 of the magnitudes, 1.4 in the mean (a library's fp32 product of the same values 191, 106).  So
// the sums stay in the instruction; the vector unit has nothing to do.
//
// A lane holds one group of a row (16 bytes), lane group g = lane / 16 the g-th of four.  Which groups of
// k make up an instruction is free as long as both operands agree: lane group g of instruction t takes
// group G g + t of a stage of 4 G, so that its G exponents are neighbouring bytes of one word, which
// the instruction selects among.  b is the instruction's first operand and a its second, so a lane's four
// results are consecutive n of one m.
#include "block_launch.h"
#include "block_types.h"
#include "gemm_tile.h"

namespace cbr {
namespace {

using namespace gemm;

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int BK = 128;     // bytes of a row in LDS: 256 values, eight groups, two words of exponents

struct Fp4Args : TileArgs {
    const uint8_t *a, *b;
    const uint32_t *sa, *sb;    // [words][M or N], a word for four groups
    int bytes;                  // of a row's groups
    int lda, ldb;
    int stages;                 // of BK bytes
    int per;                    // stages a split takes
    int words;                  // of exponents a row
};

// 16 x 16 results of four groups; S: which byte of the exponents.
template <int S>
__device__ __forceinline__ f32x4 product(u32x4 b, u32x4 a, f32x4 c, uint32_t sb, uint32_t sa)
{
    const i32x8 x = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0}, y = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, S, (int)sb, S, (int)sa);
}

// A word of exponents.  (Each lane group its own two bytes, read as such: 8 cycles of conflicts a read, as much as all
// fragments take.)
template <int OFF>
__device__ __forceinline__ uint32_t lds_word(uint32_t addr)
{
    uint32_t v;
    asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(OFF) : "memory");
    return v;
}

// Position of a row's 16-byte chunks in LDS.  A read of 16 bytes a lane goes by sixteen lanes: of each 32 lanes those of
// rows 0 to 3 and 12 to 15 with the next lane group's of rows 4 to 11, and the others.  Lane group g reads chunk 2 g
// or 2 g + 1, so rows 4 to 11 have the upper half of the positions.  (With perm() itself, which suits chunk g, each read took
// eight cycles instead of four.)
__device__ constexpr int apart(int p) { return ((p >> 2 ^ p >> 1) & 1) << 2 | (p >> 2) << 1 | (p & 1); }

// Tile kernel: 16 MS WM x 16 NS WN results a workgroup, WM x WN waves of 16 MS x 16 NS.  Both operands'
// rows of a stage and their exponents come straight into LDS, NST stages deep, as in the 8-bit product.
// 8192^3: 264 to 271 us, 4.2 to 4.1 PFLOP/s (the matrix instructions alone, from registers, 7.6), with the clock down to 2 GHz by the power it takes; of it the loads alone take
// 230 us (exponents, four bytes a lane: 17), the matrix instructions 182, the reads from LDS 90.  Smaller ones are
// bound by the way in and out of a workgroup: 50001 x 256 x 1024 17 us, of which 13 to 15 without any one of these.
template <int BM, int BN>
constexpr int word_row() { return (BM + BN) * 4 + 128; }   // words of a stage's half, 32 banks apart
template <int BM, int BN>
constexpr int stage_bytes() { return (BM + BN) * BK + 2 * word_row<BM, BN>(); }

template <int MS, int NS, int WM, int WN, int NST, bool F32>
__global__ __launch_bounds__(64 * WM * WN, 2) void gemm4_tile_kernel(Fp4Args p)
{
    constexpr int NW = WM * WN, BM = 16 * MS * WM, BN = 16 * NS * WN;
    constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;        // load instructions a wave, 8 rows each
    constexpr int LS = (BM + BN) / 64 * 2 / NW;              // of exponents, 64 rows each: of a half the waves, of b the others
    constexpr int PER = LA + LB + LS;
    constexpr int STAGE = stage_bytes<BM, BN>(), WORDS = (BM + BN) * BK, HALF = word_row<BM, BN>();
    static_assert(LA * 8 * NW == BM && LB * 8 * NW == BN && BM == BN && LS * 64 * NW == 2 * (BM + BN), "tile shape");
    static_assert(NS % 2 == 0 && MS >= 2, "products in pairs, loads at the second fragment");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const uint32_t lbase = (uint32_t)(uintptr_t)(lds_u8 *)lds;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    const int wm = wave / WN, wn = wave % WN;

    int tm, tn, split;
    place(p, tm, tn, split);
    const int64_t m0 = (int64_t)tm * BM;
    const int n0 = tn * BN;
    const int t0 = split * p.per, turns = min(p.stages, t0 + p.per) - t0;

    // rows past the end of an operand lie past the end of its buffer and read as zeros
    const int rows_a = (int)min((int64_t)BM, p.M - m0), rows_b = min(BN, p.N - n0);
    const __amdgpu_buffer_rsrc_t ra =
        __builtin_amdgcn_make_buffer_rsrc((void *)(p.a + m0 * p.lda), 0, (int)((uint32_t)rows_a * p.lda), 0x00020000);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc((void *)(p.b + (int64_t)n0 * p.ldb), 0,
                                                                        (int)((uint32_t)rows_b * p.ldb), 0x00020000);
    const int lrow = 8 * wave + (lane >> 3);
    const int lchunk = 16 * ((lane & 7) ^ apart(perm(lrow))), lchunk_b = 16 * ((lane & 7) ^ apart(perm_b<F32>(lrow)));
    // (scalars of the wave: taken by value below, where a choice between captured ones would go through memory)
    const bool of_a = wave < NW / 2;
    const int first = of_a ? wave : wave - NW / 2, s_lds = of_a ? 0 : BM * 4;
    const int s_len = 4 * (of_a ? rows_a : rows_b);
    const int64_t s_ld = of_a ? p.M : (int64_t)p.N;
    const uint32_t *const s_from = of_a ? p.sa + m0 : p.sb + n0;
    auto load = [=](int t, int st) __attribute__((always_inline)) {
        const int kat = t * BK + lchunk, kbt = t * BK + lchunk_b;   // groups past the end: zeros
        lds_u8 *base = (lds_u8 *)lds + st * STAGE;
        lds_u8 *dst = base + wave * 1024;
        const int va = kat < p.bytes ? lrow * p.lda + kat : (int)OOB, vb = kbt < p.bytes ? lrow * p.ldb + kbt : (int)OOB;
#pragma unroll
        for (int i = 0; i < LA; ++i)
            buffer_load_lds16(ra, dst + i * NW * 1024, va + i * 8 * NW * p.lda);   // (OOB and 2^30 more stays past the end)
#pragma unroll
        for (int i = 0; i < LB; ++i)
            buffer_load_lds16(rb, dst + BM * BK + i * NW * 1024, vb + i * 8 * NW * p.ldb);
#pragma unroll
        for (int i = 0; i < LS; ++i) {   // half h's words of 64 rows
            const int n = i * (NW / 2) + first, h = n / (BM / 64), at = n % (BM / 64) * 64, word = 2 * t + h;
            const __amdgpu_buffer_rsrc_t rs =
                __builtin_amdgcn_make_buffer_rsrc((void *)(s_from + word * s_ld), 0, word < p.words ? s_len : 0, 0x00020000);
            buffer_load_lds4(rs, base + WORDS + h * HALF + s_lds + at * 4, (at + lane) * 4);
        }
    };

    f32x4 acc[NS][MS];
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int j = 0; j < MS; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const uint32_t fa0 = lbase + (wm * 16 * MS + r16) * BK + 16 * (2 * g ^ apart(perm(r16)));
    const int brow = col_in_wave<F32>(0, r16 >> 2, r16 & 3);
    const uint32_t fb0 = lbase + (BM + wn * 16 * NS + brow) * BK + 16 * (2 * g ^ apart(perm_b<F32>(brow)));
    // exponents: the word with the lane's two groups, moved to its low bytes
    const uint32_t sa0 = lbase + WORDS + (g >> 1) * HALF + (wm * 16 * MS + r16) * 4;
    const uint32_t sb0 = lbase + WORDS + (g >> 1) * HALF + (BM + wn * 16 * NS + brow) * 4;
    const int shift = 16 * (g & 1);

#pragma unroll
    for (int t = 0; t < NST - 1; ++t)
        if (t < turns) load(t0 + t, t);
    int st = 0;
    for (int t = 0; t < turns; ++t) {
        vm_wait_stages<PER, NST - 2>(turns - 1 - t);
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        if (t0 + t + 1 == p.stages && (p.bytes & 63)) {
            // the word that the groups end in: what lies behind them is not used
            const int keep = (p.bytes & 63) / 16 * 8;
            uint8_t *w = lds + st * STAGE + WORDS + ((p.words - 1) & 1) * HALF;
            for (int r = threadIdx.x; r < BM + BN; r += 64 * NW) ((uint32_t *)w)[r] &= (1u << keep) - 1u;
            __syncthreads();
        }
        const uint32_t fa = fa0 + st * STAGE, fb = fb0 + st * STAGE, fax = fa ^ 16, fbx = fb ^ 16;
        const uint32_t sa = sa0 + st * STAGE, sb = sb0 + st * STAGE;
        // Products of the first instruction's fragments, then of the second's: so few are waited for at the beginning.
        // Turn q: fragment q % MS of a, instruction q / MS.
        uint32_t ea[MS], eb[NS];
        u32x4 bf[NS][2], af[3];
        auto read_a = [&](auto qc) __attribute__((always_inline)) {
            constexpr int q = decltype(qc)::value;
            if constexpr (q < 2 * MS) af[q % 3] = lds_read16<(q % MS) * 16 * BK>(q < MS ? fa : fax);
        };
        unrolled<NS>([&](auto ic) __attribute__((always_inline)) {
            constexpr int i = decltype(ic)::value;
            eb[i] = lds_word<col_in_wave<F32>(i, 0, 0) * 4>(sb);
        });
        unrolled<NS>([&](auto ic) __attribute__((always_inline)) {
            constexpr int i = decltype(ic)::value;
            bf[i][0] = lds_read16<col_in_wave<F32>(i, 0, 0) * BK>(fb);
        });
        unrolled<MS>([&](auto jc) __attribute__((always_inline)) {
            constexpr int j = decltype(jc)::value;
            ea[j] = lds_word<j * 64>(sa);
        });
        read_a(std::integral_constant<int, 0>{});
        read_a(std::integral_constant<int, 1>{});
        unrolled<2 * MS>([&](auto qc) __attribute__((always_inline)) {
            constexpr int q = decltype(qc)::value, J = q % MS, K = q / MS;
            // all but what was read after this fragment: the next one, and b's second ones behind turn 0
            lgkm_wait<(q == 1 ? NS + 1 : q == 2 * MS - 1 ? 0 : 1)>();
            if constexpr (q == 0) {
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    after_wait(eb[i]);
                    after_wait(bf[i][0]);
                    eb[i] >>= shift;
                }
#pragma unroll
                for (int j = 0; j < MS; ++j) {
                    after_wait(ea[j]);
                    ea[j] >>= shift;
                }
            }
            if constexpr (q == MS)
#pragma unroll
                for (int i = 0; i < NS; ++i) after_wait(bf[i][1]);
            after_wait(af[q % 3]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < NS; ++i) acc[i][J] = product<K>(bf[i][K], af[q % 3], acc[i][J], eb[i], ea[J]);
            if constexpr (q == 0)
                unrolled<NS>([&](auto ic) __attribute__((always_inline)) {
                    constexpr int i = decltype(ic)::value;
                    bf[i][1] = lds_read16<col_in_wave<F32>(i, 0, 0) * BK>(fbx);
                });
            // the next fragment but one, once the products that read its registers are under way
            read_a(std::integral_constant<int, q + 2>{});
            // Stage t + NST - 1 takes the place of stage t - 1, which every wave has read
            if constexpr (q == 1)
                if (t + NST - 1 < turns) load(t0 + t + NST - 1, st == 0 ? NST - 1 : st - 1);
            __builtin_amdgcn_sched_barrier(0);
        });
        st = st + 1 == NST ? 0 : st + 1;
    }
    store_tile<MS, NS, F32>(p, acc, split, m0 + wm * 16 * MS + r16, n0 + wn * 16 * NS + col_in_wave<F32>(0, g, 0));
}

// Few rows of a (m <= 16 MS): bound by reading b once.  A workgroup takes 16 columns, its eight waves share
// the runs of 512 values (256 bytes of a row: 64 by each lane group, with one word of exponents), and both
// operands come from memory straight into the instruction's registers; the waves' sums are added through
// LDS in wave order.  (1 x 1000 x 2048: 3.3 us, the launch and one round of loads; 1 x 8192 x 8192 10.4, 3.4 TB/s.  With 16
// bytes by each lane group, 64 in a row at once, and a word of exponents for each load: 12.9.)
constexpr int SKW = 8, RUN = 256;

template <int MS>
__global__ __launch_bounds__(64 * SKW) void gemm4_few_kernel(Fp4Args p)
{
    __shared__ f32x4 red[SKW][MS][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16, nl = n0 + 4 * g;
    const int t0 = blockIdx.y * p.per, t1 = min(p.stages, t0 + p.per);   // (stages of RUN bytes here)
    // rows past the end read the last one; their results are not stored
    const int nrow = min(n0 + r16, p.N - 1);
    const uint8_t *brow = p.b + (int64_t)nrow * p.ldb + 64 * g;
    const uint8_t *arow[MS];
    int mrow[MS];
#pragma unroll
    for (int j = 0; j < MS; ++j) {
        mrow[j] = min(16 * j + r16, (int)p.M - 1);
        arow[j] = p.a + (int64_t)mrow[j] * p.lda + 64 * g;
    }
    f32x4 acc[MS];
#pragma unroll
    for (int j = 0; j < MS; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    struct Run {
        u32x4 b[4], a[MS][4];
        uint32_t eb, ea[MS];
    };
    auto fetch = [&](int t, Run &o) __attribute__((always_inline)) {
        // groups past the end are zeros with the exponent 2^-127
        const int at = t * RUN, left = (p.bytes - at) / 16 - 4 * g;   // groups from this lane's first one on
        const int64_t word = 4 * t + g;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o.b[i] = i < left ? *(const u32x4 *)(brow + at + 16 * i) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int j = 0; j < MS; ++j)
                o.a[j][i] = i < left ? *(const u32x4 *)(arow[j] + at + 16 * i) : u32x4{0u, 0u, 0u, 0u};
        }
        const uint32_t keep = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << 8 * left) - 1u;
        o.eb = left > 0 ? p.sb[word * p.N + nrow] & keep : 0u;
#pragma unroll
        for (int j = 0; j < MS; ++j) o.ea[j] = left > 0 ? p.sa[word * p.M + mrow[j]] & keep : 0u;
    };
    auto multiply = [&](const Run &o) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < MS; ++j) {
            acc[j] = product<0>(o.b[0], o.a[j][0], acc[j], o.eb, o.ea[j]);
            acc[j] = product<1>(o.b[1], o.a[j][1], acc[j], o.eb, o.ea[j]);
            acc[j] = product<2>(o.b[2], o.a[j][2], acc[j], o.eb, o.ea[j]);
            acc[j] = product<3>(o.b[3], o.a[j][3], acc[j], o.eb, o.ea[j]);
        }
    };
    int t = t0 + wave;
    if (t < t1) {
        Run now, next;
        fetch(t, now);
        for (; t + SKW < t1; t += SKW) {   // the next run loads while this one is multiplied
            fetch(t + SKW, next);
            multiply(now);
            now = next;
        }
        multiply(now);
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

__global__ __launch_bounds__(256) void gemm4_join_kernel(Fp4Args p, int splits) { join_parts(p, splits); }

// ------------------------------------------------------------------------------ plan
enum Form { FEW, TILE64, TILE128, TILE256 };

struct Fp4Plan {
    Form form;
    int ms;          // FEW: 16-row tiles
    int bm, bn;
    int splits, per, stages;
};

// The form and the number of splits with the least expected time, in us, fitted to measurements of 90 shapes, each in
// all forms and with up to 13 numbers of splits: the pick takes 3% longer than the fastest in the mean, 1.2 times as
// long at worst.  Tiles: a stage of 256 values takes `one` with one workgroup on a CU and `two` with two, a
// workgroup's start and end `ends`.  Few rows: 1.2 and for each run 0.09 + 0.011 m (the more rows, the more loads), or
// b at 4.3 TB/s; two workgroups share a CU up to 16 rows.  Joining splits takes 3 to 4 us and moves each part twice at
// 4 TB/s.  (1 x 1000 x 2048: few rows 3.2 us, tiles of 64 5.6; 1 x 50000 x 512: 7.9, 6.0, tiles of 128 5.2; 64 x 256 x 50176:
// few rows 73 whole, 14.5 in 14 splits, tiles of 64 67 whole, 10.8 in 28 splits (the pick), 9.9 in 40.)
struct Costs {
    double one, two, ends;
};

Fp4Plan plan_of(const cbr_gemm_fp4_shape &s)
{
    const int64_t bytes = (s.k + 31) / 32 * 16;
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    Fp4Plan best{};
    double least = 0;
    auto weigh = [&](Form form, int64_t edge_m, int64_t edge_n, int64_t stages, int64_t fit, auto time) {
        const int64_t tiles = up(s.m, edge_m) * up(s.n, edge_n), most = tiles < fit ? std::min(fit / tiles, stages) : 1;
        for (int64_t want = 1; want <= most; want += want < 8 ? 1 : 8) {   // see place() for eights
            const int64_t per = up(stages, want), splits = up(stages, per);
            const double join = splits > 1 ? (form == FEW ? 3. : 3.5) + 0.03 * splits + (double)splits * s.m * s.n * 8. / 4e6 : 0.;
            const double t = time(per, tiles * splits) + join;
            if (best.splits == 0 || t < least) {
                least = t;
                best = Fp4Plan{form, (int)edge_m / 16, (int)edge_m, (int)edge_n, (int)splits, (int)per, (int)stages};
            }
        }
    };
    if (s.m <= 64) {
        const int64_t rows = s.m <= 16 ? 16 : s.m <= 32 ? 32 : 64;
        weigh(FEW, rows, 16, up(bytes, RUN), 512, [&](int64_t per, int64_t wgs) {
            return 2. + std::max(up(wgs, rows == 16 ? 512 : 256) * (1.2 + per * (0.09 + 0.011 * s.m)), s.n * bytes / 4.3e6 * (1. + 0.02 * s.m));
        });
    }
    for (const Form form : {TILE64, TILE128, TILE256}) {
        const Costs c = form == TILE256 ? Costs{1.0, 0., 5.} : form == TILE128 ? Costs{0.5, 0.7, 3.} : Costs{0.3, 0.35, 1.6};
        const int64_t edge = form == TILE256 ? 256 : form == TILE128 ? 128 : 64;
        weigh(form, edge, edge, up(bytes, BK), form == TILE256 ? 256 : 512, [&](int64_t per, int64_t wgs) {
            return 2.3 + (wgs <= 256 || form == TILE256 ? up(wgs, 256) * (per * c.one + c.ends) : up(wgs, 512) * (per * c.two + c.ends));
        });
    }
    return best;
}

template <int MS, int NS, int WM, int WN, int NST, bool F32>
hipError_t launch_tile(const Fp4Args &a, hipStream_t st)
{
    auto k = gemm4_tile_kernel<MS, NS, WM, WN, NST, F32>;
    constexpr int lds = NST * stage_bytes<16 * MS * WM, 16 * NS * WN>();
    static_assert(lds <= 160 * 1024, "LDS of a CU");
    const hipError_t e = raise_lds_limit((const void *)k, lds);
    if (e != hipSuccess) return e;
    return launch(k, dim3((uint32_t)a.tiles_m * a.tiles_n * a.splits), dim3(64 * WM * WN), lds, st, nullptr, nullptr, a);
}

template <bool F32>
hipError_t launch_form(const Fp4Plan &pl, const Fp4Args &a, hipStream_t st)
{
    if (pl.form == TILE256) return launch_tile<8, 4, 2, 4, 2, F32>(a, st);
    if (pl.form == TILE64) return launch_tile<2, 2, 2, 2, 4, F32>(a, st);
    // one workgroup a CU: four stages deep; more: two, and two workgroups share a CU
    return (int64_t)a.tiles_m * a.tiles_n * pl.splits <= 256 ? launch_tile<4, 2, 2, 4, 4, F32>(a, st)
                                                             : launch_tile<4, 4, 2, 2, 2, F32>(a, st);
}

}  // namespace

size_t gemm_fp4_part_bytes(const cbr_gemm_fp4_shape &s)
{
    const Fp4Plan p = plan_of(s);
    return p.splits > 1 ? (size_t)p.splits * s.m * s.n * sizeof(float) : 0;
}

hipError_t launch_gemm_fp4(const cbr_gemm_fp4_shape &s, const void *a, const void *a_scale, const void *b,
                           const void *b_scale, const float *bias, void *d, float *part, hipStream_t st)
{
    const Fp4Plan pl = plan_of(s);
    Fp4Args p{};
    p.a = (const uint8_t *)a;
    p.b = (const uint8_t *)b;
    p.sa = (const uint32_t *)a_scale;
    p.sb = (const uint32_t *)b_scale;
    p.bias = bias;
    p.d = d;
    p.part = pl.splits > 1 ? part : nullptr;
    p.M = s.m;
    p.N = (int)s.n;
    p.bytes = (int)((s.k + 31) / 32 * 16);
    p.lda = (int)s.lda;
    p.ldb = (int)s.ldb;
    p.stages = pl.stages;
    p.per = pl.per;
    p.words = (int)((s.k + 127) / 128);
    p.d_type = s.d_type;
    p.relu = s.relu;
    p.splits = pl.splits;
    p.tiles_m = (int)((s.m + pl.bm - 1) / pl.bm);
    p.tiles_n = (int)((s.n + pl.bn - 1) / pl.bn);
    hipError_t e;
    if (pl.form == FEW) {
        auto k = pl.ms == 1 ? gemm4_few_kernel<1> : pl.ms == 2 ? gemm4_few_kernel<2> : gemm4_few_kernel<4>;
        e = launch(k, dim3(p.tiles_n, pl.splits), dim3(64 * SKW), 0, st, nullptr, nullptr, p);
    } else {
        e = s.d_type == CBR_F32 ? launch_form<true>(pl, p, st) : launch_form<false>(pl, p, st);
    }
    if (e != hipSuccess || pl.splits == 1) return e;
    const int64_t quads = s.m * ((s.n + 3) / 4);
    return launch(gemm4_join_kernel, dim3((uint32_t)((quads + 255) / 256)), dim3(256), 0, st, nullptr, nullptr, p, pl.splits);
}

}  // namespace cbr
