// block_norm_fwd.hip -- the residual add around a block with the norms on both its sides:
//   n = post(f),  y = x + alpha r g n,  h = pre(y)
// in one pass over x and f.  A row's values stay in registers from the load to the last
// store, so each norm takes its mean first and the squared deviations after it (no
// difference of large sums), and y goes into the second norm before it is rounded.
// Bound by memory: x and f are read once, y and h written once (200704 x 512 bf16: 162 us =
// 5.1 TB/s, of 5.2 that a copy reaches; 49 x 512: 3.7 us, a launch and one row's sums).
#include "block_norm.h"

namespace cbr {
namespace {

using namespace bnorm;

constexpr int E = 8;   // values a thread (sixteen with their coefficients do not fit 128 registers)

// (v - mean) / std of a row in place; st: (mean, 1/std).
template <Tail TAIL>
__device__ __forceinline__ void normalise(float (&v)[E], int kind, float eps, int l, int L, int C, RowSum<1> &sum,
                                          float &mean, float &inv)
{
    mean = 0.f;
    if (kind == CBR_NORM_LAYER) {
        float s[1] = {0.f};
#pragma unroll
        for (int j = 0; j < E; ++j) s[0] += v[j];
        sum(s);
        mean = s[0] / (float)C;
#pragma unroll
        for (int j = 0; j < E; ++j)
            if (has<E, TAIL>(j, l, L, C)) v[j] -= mean;   // the values past the row stay 0
    }
    float q[1] = {0.f};
#pragma unroll
    for (int j = 0; j < E; ++j) q[0] = fmaf(v[j], v[j], q[0]);
    sum(q);
    inv = 1.f / sqrtf(q[0] / (float)C + eps);
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] *= inv;
}

template <typename TS, typename TB, Tail TAIL>
__global__ __launch_bounds__(1024) void block_norm_fwd_kernel(BlockNormArgs p, int L, int rpb)
{
    __shared__ float red[2][MAX_WAVES][1];
    RowSum<1> sum{red, L, 0};
    const int C = p.C, l = threadIdx.x % L, sub = threadIdx.x / L;
    const uint32_t step = gridDim.x * rpb;
    // every thread of the workgroup takes the same number of turns (the sums may hold a barrier)
    const uint32_t turns = (p.rows - blockIdx.x * rpb + step - 1) / step;   // blockIdx.x * rpb < rows
    Row<TS, E, TAIL> xn;
    Row<TB, E, TAIL> fn;
    auto fetch = [&](uint64_t row) __attribute__((always_inline)) {
        const bool on = row < p.rows;
        xn.load((const char *)p.x + row * C * TS::SIZE, l, L, C, on);
        fn.load((const char *)p.f + row * C * TB::SIZE, l, L, C, on && p.f);
    };
    uint64_t row = (uint64_t)blockIdx.x * rpb + sub;
    fetch(row);   // with the vectors: one latency of memory
    // y = x + g (cw nhat + cb), h = pw yhat + pb
    float cw[E], cb[E], pw[E], pb[E];
    {
        float r[E];
        load_vec<E, TAIL>(p.res_scale, 1.f, l, L, C, r);
        load_vec<E, TAIL>(p.post_w, 1.f, l, L, C, cw);
        load_vec<E, TAIL>(p.post_b, 0.f, l, L, C, cb);
#pragma unroll
        for (int j = 0; j < E; ++j) {
            cw[j] *= p.alpha * r[j];
            cb[j] *= p.alpha * r[j];
        }
    }
    load_vec<E, TAIL>(p.pre_w, 1.f, l, L, C, pw);
    load_vec<E, TAIL>(p.pre_b, 0.f, l, L, C, pb);
    for (uint32_t t = 0; t < turns; ++t, row += step) {
        float v[E], y[E];
        xn.get(y, l, L, C);
        fn.get(v, l, L, C);
        const bool on = row < p.rows;
        Row<TB, E, TAIL> g;
        if (p.gate)
            g.load((const char *)p.gate + (uint64_t)((uint32_t)row / p.rpg) * C * TB::SIZE, l, L, C, on);
        if (t + 1 < turns) fetch(row + step);   // the next row's loads run beside this row's sums
        float mean, inv;
        if (p.f) {
            if (p.post != CBR_NORM_NONE) {
                normalise<TAIL>(v, p.post, p.eps_post, l, L, C, sum, mean, inv);
                if (on && l == 0 && p.post_stats) *(f32x2 *)(p.post_stats + 2 * row) = f32x2{mean, inv};
            }
            if (p.gate) {
                float gv[E];
                g.get(gv, l, L, C);
#pragma unroll
                for (int j = 0; j < E; ++j) y[j] = fmaf(gv[j], fmaf(cw[j], v[j], cb[j]), y[j]);
            } else {
#pragma unroll
                for (int j = 0; j < E; ++j) y[j] += fmaf(cw[j], v[j], cb[j]);
            }
            if (on) Row<TS, E, TAIL>::store((char *)p.y + row * C * TS::SIZE, l, L, C, y);
        }
        if (p.pre != CBR_NORM_NONE) {
            normalise<TAIL>(y, p.pre, p.eps_pre, l, L, C, sum, mean, inv);
            if (on && l == 0 && p.pre_stats) *(f32x2 *)(p.pre_stats + 2 * row) = f32x2{mean, inv};
#pragma unroll
            for (int j = 0; j < E; ++j) y[j] = fmaf(pw[j], y[j], pb[j]);
            if (on) Row<TB, E, TAIL>::store((char *)p.h + row * C * TB::SIZE, l, L, C, y);
        }
    }
}

template <typename TS, typename TB>
hipError_t launch_types(const BlockNormArgs &a, hipStream_t st)
{
    const Layout o = layout_of(a.C, 256, 1024);
    const uint32_t need = (uint32_t)(((uint64_t)a.rows + o.rpb - 1) / o.rpb);
    // As many workgroups as run at once (sixteen waves a CU), each with the same number of rows
    const uint32_t most = 256u * std::max(1u, 1024u / o.threads), turns = (need + most - 1) / most;
    const uint32_t grid = (need + turns - 1) / turns;
    auto k = o.tail == WHOLE  ? block_norm_fwd_kernel<TS, TB, WHOLE>
             : o.tail == PART ? block_norm_fwd_kernel<TS, TB, PART> : block_norm_fwd_kernel<TS, TB, SHORT>;
    return launch(k, dim3(grid), dim3(o.threads), 0, st, nullptr, nullptr, a, o.L, o.rpb);
}

}  // namespace

hipError_t launch_block_norm_fwd(const BlockNormArgs &a, int stream_type, int branch_type, hipStream_t st)
{
    if (stream_type == CBR_BF16) return launch_types<Bf16, Bf16>(a, st);
    if (stream_type == CBR_F16) return launch_types<F16, F16>(a, st);
    if (branch_type == CBR_BF16) return launch_types<F32, Bf16>(a, st);
    if (branch_type == CBR_F16) return launch_types<F32, F16>(a, st);
    return launch_types<F32, F32>(a, st);
}

}  // namespace cbr
