// block_launch.h -- host-side plan and launch functions of the block norm, the 8-bit
// quantiser and the 8-bit matrix product (internal).
#pragma once

#include "../../include/cbr.h"
#include "cbr_launch.h"

namespace cbr {

// The block norm's operands as the kernels see them (include/cbr.h has their meaning).
struct BlockNormArgs {
    uint32_t rows, rpg;        // rpg: rows of a gate row (rows where there is no gate)
    int C;
    int post, pre;             // enum cbr_norm
    float alpha, eps_post, eps_pre;
    const void *x, *f, *gate;  // x: y in the backward
    const float *post_w, *post_b, *res_scale, *pre_w, *pre_b;
    void *y, *h;
    float *post_stats, *pre_stats;
    // backward
    const void *dy, *dh;
    void *dx, *df, *dgate;
    float *dpost_w, *dpost_b, *dres_scale, *dpre_w, *dpre_b;
    float *part;               // the workgroups' partial sums over rows
};

hipError_t launch_block_norm_fwd(const BlockNormArgs &a, int stream_type, int branch_type, hipStream_t st);
// Bytes of the backward's partial sums, with or without a gate (rpg 0: without).
size_t block_norm_part_bytes(uint32_t rows, uint32_t rpg, int C);
hipError_t launch_block_norm_bwd(const BlockNormArgs &a, int stream_type, int branch_type, hipStream_t st);

hipError_t launch_fp8_quantize(const cbr_quant_shape &s, const void *src, void *q, float *scale, hipStream_t st);

size_t gemm_fp8_part_bytes(const cbr_gemm_shape &s);
hipError_t launch_gemm_fp8(const cbr_gemm_shape &s, const void *a, const float *a_scale, const void *b,
                           const float *b_scale, const float *bias, void *d, float *part, hipStream_t st);

}  // namespace cbr
