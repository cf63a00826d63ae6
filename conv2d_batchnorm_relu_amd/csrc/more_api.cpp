// more_api.cpp -- C ABI of the group norm, the 4-bit quantiser and the 4-bit matrix product: argument
// validation and launches.  As in cbr_api.cpp, everything is checked on the host before the first HIP call.
#include <math.h>

#include <algorithm>

#include "../../include/cbr.h"
#include "block_launch.h"
#include "group_norm.h"

using namespace cbr;

namespace {

constexpr int64_t MAX_ROWS = 2147483647;
constexpr int32_t MAX_GROUP = 8192;        // channels of a group: 1024 threads of eight
constexpr int64_t MAX_STRIDE = 1 << 22;    // 256 rows of a product's tile stay within 31-bit byte offsets
constexpr int64_t MAX_K = 1 << 23;
constexpr int64_t MAX_GROUPS = 1 << 24;    // workgroups of 256 threads: a launch holds fewer than 2^32 threads

template <typename... T>
bool all_aligned(T... ps)
{
    return ((((uintptr_t)ps & 15u) == 0) && ...);   // NULL is aligned
}

bool float_type(int32_t t) { return t == CBR_BF16 || t == CBR_F16 || t == CBR_F32; }

// Checks the shape and lays the call out.
int check_group_norm(const cbr_group_norm_shape *s, bool backward, gnorm::Geo &g)
{
    if (!s) return CBR_E_NULL;
    if (s->images <= 0 || s->pixels <= 0 || s->channels <= 0 || s->groups <= 0 || s->channels % s->groups) return CBR_E_SHAPE;
    if (!float_type(s->type) || (s->act != CBR_ACT_NONE && s->act != CBR_ACT_RELU && s->act != CBR_ACT_SILU) || !(s->eps >= 0.f) ||
        !isfinite(s->eps))
        return CBR_E_VALUE;
    if (s->images > MAX_ROWS || s->pixels > MAX_ROWS || s->channels / s->groups > MAX_GROUP || s->channels >= 1 << 24) return CBR_E_UNSUPPORTED;
    // within 2^46 values nothing below overflows; a launch holds fewer than 2^32 threads
    if ((double)s->images * (double)s->pixels * s->channels > 0x1p46) return CBR_E_UNSUPPORTED;
    g = gnorm::plan_group_norm(*s, backward);
    // (and the workgroups of 16 channels before those of the images in the backward's last kernel)
    return (gnorm::workgroups(*s, g) + s->channels / 16 + 1) * gnorm::threads_of(g) < (int64_t)1 << 32 ? CBR_OK : CBR_E_UNSUPPORTED;
}

// Workspace bytes, rounded up.
size_t norm_bytes(const cbr_group_norm_shape *s, const gnorm::Geo &g, bool backward)
{
    return (gnorm::part_bytes(*s, g, backward) + 255) / 256 * 256;
}

int check_fp4(const cbr_fp4_shape *s)
{
    if (!s) return CBR_E_NULL;
    if (s->rows <= 0 || s->cols <= 0) return CBR_E_SHAPE;
    if (!float_type(s->type)) return CBR_E_VALUE;
    if (s->rows > MAX_ROWS || s->cols > MAX_ROWS) return CBR_E_UNSUPPORTED;
    const int64_t v_cols = s->transpose ? s->rows : s->cols;
    if (s->ldq < (v_cols + 31) / 32 * 16 || s->ldq % 16) return CBR_E_SHAPE;
    // a workgroup for each 16 rows and 128 columns of v, or more of them
    const int64_t v_rows = s->transpose ? s->cols : s->rows;
    if (((v_rows + 15) / 16) * ((v_cols + 127) / 128) >= MAX_GROUPS) return CBR_E_UNSUPPORTED;
    return CBR_OK;
}

int check_gemm4(const cbr_gemm_fp4_shape *s)
{
    if (!s) return CBR_E_NULL;
    if (s->m <= 0 || s->n <= 0 || s->k <= 0) return CBR_E_SHAPE;
    if (!float_type(s->d_type)) return CBR_E_VALUE;
    if (s->k > MAX_K) return CBR_E_UNSUPPORTED;
    const int64_t bytes = (s->k + 31) / 32 * 16;
    if (s->lda < bytes || s->ldb < bytes || s->lda % 16 || s->ldb % 16) return CBR_E_SHAPE;
    if (s->m > MAX_ROWS || s->n > MAX_STRIDE || s->lda > MAX_STRIDE || s->ldb > MAX_STRIDE) return CBR_E_UNSUPPORTED;
    // workgroups of 256 threads for 64 x 64 results, of 512 for 128 x 128 (one row of tiles: half as many, rounded up)
    if (((s->m + 63) / 64) * ((s->n + 63) / 64) >= MAX_GROUPS - 1) return CBR_E_UNSUPPORTED;
    return CBR_OK;
}

gnorm::GroupNormArgs norm_args(const cbr_group_norm_shape *s, const gnorm::Geo &g)
{
    gnorm::GroupNormArgs a{};
    a.g = g;
    a.nt = gnorm::streams(*s, g);
    a.images = s->images;
    a.pixels = s->pixels;
    a.C = s->channels;
    a.G = s->groups;
    a.cpg = s->channels / s->groups;
    a.act = s->act;
    a.eps = s->eps;
    return a;
}

}  // namespace

extern "C" {

size_t cbr_group_norm_workspace_bytes(const cbr_group_norm_shape *shape, int backward)
{
    gnorm::Geo g;
    return check_group_norm(shape, backward != 0, g) == CBR_OK ? norm_bytes(shape, g, backward != 0) : 0;
}

int cbr_group_norm_forward(const cbr_group_norm_shape *shape, const void *x, const float *w, const float *b, void *y,
                           float *stats, void *workspace, size_t ws_bytes, void *stream)
{
    gnorm::Geo g;
    const int st = check_group_norm(shape, false, g);
    if (st != CBR_OK) return st;
    if (!x || !y) return CBR_E_NULL;
    if (!all_aligned(x, w, b, y, stats)) return CBR_E_ALIGN;
    const size_t need = norm_bytes(shape, g, false);
    if (need && (!workspace || ws_bytes < need)) return CBR_E_WORKSPACE;
    if (need && !all_aligned(workspace)) return CBR_E_ALIGN;
    gnorm::GroupNormArgs a = norm_args(shape, g);
    a.x = x;
    a.w = w;
    a.b = b;
    a.out = y;
    a.stats = stats;
    a.part = need ? (float *)workspace : nullptr;
    return launch_group_norm_fwd(*shape, a, (hipStream_t)stream) == hipSuccess ? CBR_OK : CBR_E_HIP;
}

int cbr_group_norm_backward(const cbr_group_norm_shape *shape, const void *dy, const void *x, const float *w, const float *b,
                            const float *stats, void *dx, float *dw, float *db, void *workspace, size_t ws_bytes, void *stream)
{
    gnorm::Geo g;
    const int st = check_group_norm(shape, true, g);
    if (st != CBR_OK) return st;
    if (!dy || !x || !stats || (!dx && !dw && !db)) return CBR_E_NULL;
    if (!all_aligned(dy, x, w, b, stats, dx, dw, db)) return CBR_E_ALIGN;
    const size_t need = norm_bytes(shape, g, true);
    if (need && (!workspace || ws_bytes < need)) return CBR_E_WORKSPACE;
    if (need && !all_aligned(workspace)) return CBR_E_ALIGN;
    gnorm::GroupNormArgs a = norm_args(shape, g);
    a.dy = dy;
    a.x = x;
    a.w = w;
    a.b = b;
    a.stats_in = stats;
    a.out = dx;
    a.dw = dw;
    a.db = db;
    a.part = need ? (float *)workspace : nullptr;
    return launch_group_norm_bwd(*shape, a, (hipStream_t)stream) == hipSuccess ? CBR_OK : CBR_E_HIP;
}

int cbr_fp4_quantize(const cbr_fp4_shape *shape, const void *src, void *q, void *scale, void *stream)
{
    const int st = check_fp4(shape);
    if (st != CBR_OK) return st;
    if (!src || !q || !scale) return CBR_E_NULL;
    if (!all_aligned(src, q, scale)) return CBR_E_ALIGN;
    return launch_fp4_quantize(*shape, src, q, scale, (hipStream_t)stream) == hipSuccess ? CBR_OK : CBR_E_HIP;
}

int cbr_fp4_dequantize(const cbr_fp4_shape *shape, const void *q, const void *scale, void *v, void *stream)
{
    const int st = check_fp4(shape);
    if (st != CBR_OK) return st;
    if (!q || !scale || !v) return CBR_E_NULL;
    if (!all_aligned(q, scale, v)) return CBR_E_ALIGN;
    return launch_fp4_dequantize(*shape, q, scale, v, (hipStream_t)stream) == hipSuccess ? CBR_OK : CBR_E_HIP;
}

size_t cbr_gemm_fp4_workspace_bytes(const cbr_gemm_fp4_shape *shape)
{
    if (check_gemm4(shape) != CBR_OK) return 0;
    return (gemm_fp4_part_bytes(*shape) + 255) / 256 * 256;
}

int cbr_gemm_fp4(const cbr_gemm_fp4_shape *shape, const void *a, const void *a_scale, const void *b, const void *b_scale,
                 const float *bias, void *d, void *workspace, size_t ws_bytes, void *stream)
{
    const int st = check_gemm4(shape);
    if (st != CBR_OK) return st;
    if (!a || !a_scale || !b || !b_scale || !d) return CBR_E_NULL;
    if (!all_aligned(a, a_scale, b, b_scale, bias, d)) return CBR_E_ALIGN;
    const size_t need = cbr_gemm_fp4_workspace_bytes(shape);
    if (need && (!workspace || ws_bytes < need)) return CBR_E_WORKSPACE;
    if (need && !all_aligned(workspace)) return CBR_E_ALIGN;
    return launch_gemm_fp4(*shape, a, a_scale, b, b_scale, bias, d, (float *)workspace, (hipStream_t)stream) == hipSuccess ? CBR_OK
                                                                                                                       : CBR_E_HIP;
}

}  // extern "C"
