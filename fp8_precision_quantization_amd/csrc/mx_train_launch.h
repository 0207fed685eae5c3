// Internal launchers behind mxtrain.h (arguments already validated).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx {

// Layer norm.  vec: x, w, b and the output 16-byte aligned, cols and the
// leading dimensions multiples of 8 (bf16) or 4 (binary32).
hipError_t launch_norm_fwd(const void* x, int64_t ldx, bool x_f32, const void* w, const void* b, bool w_f32,
                           int64_t rows, int64_t cols, float eps, void* y, float* mean, float* rstd, uint8_t* q,
                           uint8_t* s, bool vec, hipStream_t stream);
hipError_t launch_norm_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, bool x_f32, const void* w,
                           bool w_f32, const float* mean, const float* rstd, int64_t rows, int64_t cols, void* dx,
                           float* dw, float* db, float* part, bool vec, hipStream_t stream);
// Rows (of dw and of db sums each) that launch_norm_bwd leaves in part, at most.
int64_t norm_bwd_part_rows(int64_t rows);

// MoE router.  vec: 16-byte aligned logits (and dlogits), experts and ld
// multiples of a 16-byte word's elements.
hipError_t launch_router_fwd(const void* logits, int64_t ld, bool f32, const uint8_t* valid, int64_t rows,
                             int32_t experts, int32_t topk, bool normalize, int32_t align, int32_t* chosen,
                             float* gates, float* lse, int32_t* counts, int32_t* ends, float* balance, float* loss,
                             void* workspace, bool vec, hipStream_t stream);
int64_t router_workspace_bytes(int64_t rows, int64_t experts);
hipError_t launch_router_bwd(const void* logits, int64_t ld, bool f32, const float* lse, const int32_t* chosen,
                             const float* gates, const float* balance, const float* dgates, const float* dloss,
                             int64_t rows, int32_t experts, int32_t topk, bool normalize, void* dlogits, bool vec,
                             hipStream_t stream);

// Gated activation (q and s both null: no checkpoint; y null in the backward
// pass: not formed again).
hipError_t launch_act_fwd(const void* h, int64_t rows, int64_t cols, bool gelu, void* y, uint8_t* q, uint8_t* s,
                          hipStream_t stream);
hipError_t launch_act_bwd(const void* dy, const uint8_t* q, const uint8_t* s, int64_t rows, int64_t cols, bool gelu,
                          void* dh, void* y, hipStream_t stream);

// Weight gradient from a checkpoint.  vec: dy 16-byte aligned, lddy a
// multiple of 8.  ends null: one group.
hipError_t launch_wgrad(const void* dy, int64_t lddy, const uint8_t* q, const uint8_t* s, int64_t rows, int64_t n,
                        int64_t k, const int32_t* ends, int32_t groups, void* dw, bool bf16, float* workspace,
                        bool vec, hipStream_t stream);
int64_t wgrad_workspace_bytes(int64_t rows, int64_t n, int64_t k, int32_t groups);
int64_t wgrad_grid_blocks(int64_t rows, int64_t n, int64_t k, int32_t groups);

}  // namespace mx
