// block_api.cpp -- C ABI of the block norm, the 8-bit quantiser and the 8-bit matrix
// product: argument validation and launches.  As in cbr_api.cpp, everything is checked on
// the host before the first HIP call.
#include <math.h>

#include <algorithm>

#include "../../include/cbr.h"
#include "block_launch.h"

using namespace cbr;

namespace {

constexpr int64_t MAX_ROWS = 2147483647;
constexpr int32_t MAX_CHANNELS = 8192;     // 1024 threads of eight values
constexpr int64_t MAX_STRIDE = 1 << 23;    // 256 rows of a product's tile stay within 31-bit byte offsets
constexpr int64_t MAX_GROUPS = 1 << 24;    // workgroups of 256 threads: a launch holds fewer than 2^32 threads

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }   // NULL is aligned

template <typename... T>
bool all_aligned(T... ps)
{
    return (aligned16(ps) && ...);
}

bool float_type(int32_t t) { return t == CBR_BF16 || t == CBR_F16 || t == CBR_F32; }
bool fp8_type(int32_t t) { return t == CBR_E4M3 || t == CBR_E5M2; }
bool norm_kind(int32_t k) { return k == CBR_NORM_NONE || k == CBR_NORM_RMS || k == CBR_NORM_LAYER; }
bool eps_ok(float e) { return e >= 0.f && isfinite(e); }

int check_block(const cbr_block_shape *s)
{
    if (!s) return CBR_E_NULL;
    if (s->rows <= 0 || s->channels <= 0) return CBR_E_SHAPE;
    if (!norm_kind(s->post) || !norm_kind(s->pre) || !float_type(s->stream_type) || !float_type(s->branch_type) ||
        !isfinite(s->alpha) || !eps_ok(s->eps_post) || !eps_ok(s->eps_pre))
        return CBR_E_VALUE;
    if (s->rows > MAX_ROWS || s->channels > MAX_CHANNELS ||
        (s->stream_type != s->branch_type && s->stream_type != CBR_F32))
        return CBR_E_UNSUPPORTED;
    return CBR_OK;
}

bool gate_rows_ok(const cbr_block_shape *s) { return s->rows_per_gate > 0 && s->rows % s->rows_per_gate == 0; }

BlockNormArgs norm_args(const cbr_block_shape *s)
{
    BlockNormArgs a{};
    a.rows = (uint32_t)s->rows;
    a.rpg = gate_rows_ok(s) ? (uint32_t)s->rows_per_gate : (uint32_t)s->rows;
    a.C = s->channels;
    a.post = s->post;
    a.pre = s->pre;
    a.alpha = s->alpha;
    a.eps_post = s->eps_post;
    a.eps_pre = s->eps_pre;
    return a;
}

int check_quant(const cbr_quant_shape *s)
{
    if (!s) return CBR_E_NULL;
    if (s->rows <= 0 || s->cols <= 0) return CBR_E_SHAPE;
    if (!float_type(s->src_type) || !fp8_type(s->q_type) || (s->block != 1 && s->block != 128)) return CBR_E_VALUE;
    if (s->rows > MAX_ROWS || s->cols > MAX_ROWS) return CBR_E_UNSUPPORTED;
    const int64_t v_cols = s->transpose ? s->rows : s->cols;
    if (s->ldq < v_cols || s->ldq % 16) return CBR_E_SHAPE;
    // one workgroup for each 64 rows and 128 columns (16 rows only where there are few)
    if (((s->rows + 63) / 64) * ((s->cols + 127) / 128) >= MAX_GROUPS) return CBR_E_UNSUPPORTED;
    return CBR_OK;
}

int check_gemm(const cbr_gemm_shape *s)
{
    if (!s) return CBR_E_NULL;
    if (s->m <= 0 || s->n <= 0 || s->k <= 0) return CBR_E_SHAPE;
    if (!fp8_type(s->a_type) || !fp8_type(s->b_type) || !float_type(s->d_type) || (s->b_block != 1 && s->b_block != 128) ||
        (s->short_sums && s->d_type == CBR_F32))
        return CBR_E_VALUE;
    if (s->lda < s->k || s->ldb < s->k || s->lda % 16 || s->ldb % 16) return CBR_E_SHAPE;
    if (s->m > MAX_ROWS || s->n > MAX_STRIDE || s->lda > MAX_STRIDE || s->ldb > MAX_STRIDE)
        return CBR_E_UNSUPPORTED;
    // workgroups of 256 threads for 64 x 64 results, of 512 for 128 x 128 (one row of tiles: half as many, rounded up)
    if (((s->m + 63) / 64) * ((s->n + 63) / 64) >= MAX_GROUPS - 1) return CBR_E_UNSUPPORTED;
    return CBR_OK;
}

}  // namespace

extern "C" {

size_t cbr_block_norm_workspace_bytes(const cbr_block_shape *shape)
{
    if (check_block(shape) != CBR_OK) return 0;
    const size_t bytes =
        block_norm_part_bytes((uint32_t)shape->rows, gate_rows_ok(shape) ? (uint32_t)shape->rows_per_gate : 0u, shape->channels);
    return (bytes + 255) / 256 * 256;
}

int cbr_block_norm_forward(const cbr_block_shape *shape, const void *x, const void *f, const float *post_w,
                           const float *post_b, const void *gate, const float *res_scale, const float *pre_w,
                           const float *pre_b, void *y, void *h, float *post_stats, float *pre_stats, void *stream)
{
    const int st = check_block(shape);
    if (st != CBR_OK) return st;
    const bool post = shape->post != CBR_NORM_NONE, pre = shape->pre != CBR_NORM_NONE;
    if (!x || (f && !y) || (pre && !h)) return CBR_E_NULL;
    if ((!f && (post || gate || res_scale || y)) || (!post && (post_w || post_b || post_stats)) ||
        (!pre && (pre_w || pre_b || h || pre_stats)) || (!f && !pre))
        return CBR_E_VALUE;
    if (!all_aligned(x, f, gate) || !all_aligned(post_w, post_b, res_scale, pre_w, pre_b, post_stats, pre_stats) ||
        !all_aligned(y, h))
        return CBR_E_ALIGN;
    if (gate && !gate_rows_ok(shape)) return CBR_E_SHAPE;
    BlockNormArgs a = norm_args(shape);
    a.x = x;
    a.f = f;
    a.gate = gate;
    a.post_w = post_w;
    a.post_b = post_b;
    a.res_scale = res_scale;
    a.pre_w = pre_w;
    a.pre_b = pre_b;
    a.y = y;
    a.h = h;
    a.post_stats = post_stats;
    a.pre_stats = pre_stats;
    return launch_block_norm_fwd(a, shape->stream_type, shape->branch_type, (hipStream_t)stream) == hipSuccess ? CBR_OK
                                                                                                               : CBR_E_HIP;
}

int cbr_block_norm_backward(const cbr_block_shape *shape, const void *dy, const void *dh, const void *y, const void *f,
                            const float *post_w, const float *post_b, const void *gate, const float *res_scale,
                            const float *pre_w, const float *post_stats, const float *pre_stats, void *dx, void *df,
                            float *dpost_w, float *dpost_b, void *dgate, float *dres_scale, float *dpre_w,
                            float *dpre_b, void *workspace, size_t ws_bytes, void *stream)
{
    const int st = check_block(shape);
    if (st != CBR_OK) return st;
    const bool post = shape->post != CBR_NORM_NONE, pre = shape->pre != CBR_NORM_NONE;
    if (!dx || (pre && (!dh || !y || !pre_stats)) || (!pre && !dy) || (f && !df) || (post && (!f || !post_stats)))
        return CBR_E_NULL;
    if ((!f && (gate || res_scale || df || dres_scale)) || (!post && (post_w || post_b || post_stats || dpost_w || dpost_b)) ||
        (!pre && (pre_w || dh || pre_stats || dpre_w || dpre_b)) || (dgate && !gate) || (!f && !pre))
        return CBR_E_VALUE;
    if (!all_aligned(dy, dh, y, f, gate) || !all_aligned(post_w, post_b, res_scale, pre_w, post_stats, pre_stats) ||
        !all_aligned(dx, df, dgate) || !all_aligned(dpost_w, dpost_b, dres_scale, dpre_w, dpre_b))
        return CBR_E_ALIGN;
    if (gate && !gate_rows_ok(shape)) return CBR_E_SHAPE;
    if (!workspace || ws_bytes < cbr_block_norm_workspace_bytes(shape)) return CBR_E_WORKSPACE;
    if (!aligned16(workspace)) return CBR_E_ALIGN;
    BlockNormArgs a = norm_args(shape);
    a.dy = dy;
    a.dh = dh;
    a.x = y;
    a.f = f;
    a.post_w = post_w;
    a.post_b = post_b;
    a.gate = gate;
    a.res_scale = res_scale;
    a.pre_w = pre_w;
    a.post_stats = const_cast<float *>(post_stats);
    a.pre_stats = const_cast<float *>(pre_stats);
    a.dx = dx;
    a.df = df;
    a.dgate = dgate;
    a.dpost_w = dpost_w;
    a.dpost_b = dpost_b;
    a.dres_scale = dres_scale;
    a.dpre_w = dpre_w;
    a.dpre_b = dpre_b;
    a.part = (float *)workspace;
    return launch_block_norm_bwd(a, shape->stream_type, shape->branch_type, (hipStream_t)stream) == hipSuccess ? CBR_OK
                                                                                                               : CBR_E_HIP;
}

int cbr_fp8_quantize(const cbr_quant_shape *shape, const void *src, void *q, float *scale, void *stream)
{
    const int st = check_quant(shape);
    if (st != CBR_OK) return st;
    if (!src || !q || !scale) return CBR_E_NULL;
    if (!all_aligned(src, q, scale)) return CBR_E_ALIGN;
    return launch_fp8_quantize(*shape, src, q, scale, (hipStream_t)stream) == hipSuccess ? CBR_OK : CBR_E_HIP;
}

size_t cbr_gemm_fp8_workspace_bytes(const cbr_gemm_shape *shape)
{
    if (check_gemm(shape) != CBR_OK) return 0;
    return (gemm_fp8_part_bytes(*shape) + 255) / 256 * 256;
}

int cbr_gemm_fp8(const cbr_gemm_shape *shape, const void *a, const float *a_scale, const void *b, const float *b_scale,
                 const float *bias, void *d, void *workspace, size_t ws_bytes, void *stream)
{
    const int st = check_gemm(shape);
    if (st != CBR_OK) return st;
    if (!a || !a_scale || !b || !b_scale || !d) return CBR_E_NULL;
    if (!all_aligned(a, a_scale, b, b_scale, bias, d)) return CBR_E_ALIGN;
    const size_t need = cbr_gemm_fp8_workspace_bytes(shape);
    if (need && (!workspace || ws_bytes < need)) return CBR_E_WORKSPACE;
    if (need && !aligned16(workspace)) return CBR_E_ALIGN;
    return launch_gemm_fp8(*shape, a, a_scale, b, b_scale, bias, d, (float *)workspace, (hipStream_t)stream) == hipSuccess
               ? CBR_OK
               : CBR_E_HIP;
}

}  // extern "C"
