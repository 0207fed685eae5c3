// Internal launchers behind mxfp4.h (arguments already validated).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx {

// Operands of a product: codes and blocked scales of X (rows of the result)
// and of W (its columns, group by group).  ends null: one group.
struct MmOperands {
  const uint8_t *qx, *sx;
  int32_t x_format;
  const uint8_t *qw, *sw;
  int32_t w_format;
  const int32_t* ends;
  int32_t groups;
};

// MXFP4 cast of `batch` (rows, cols) matrices, rows ldx apart and matrices one
// after another; q0/s0 (dim0) and/or q1/s1 (dim1) non-null.
hipError_t launch_cast4(const void* x, int64_t batch, int64_t rows, int64_t cols, int64_t ldx, bool f32, uint8_t* q0,
                        uint8_t* s0, uint8_t* q1, uint8_t* s1, bool blocked, hipStream_t stream);
hipError_t launch_dequantize4(const uint8_t* q, const uint8_t* s, int64_t batch, int64_t rows, int64_t cols,
                              bool blocked, void* x, bool f32, hipStream_t stream);

hipError_t launch_gemm4(const MmOperands& in, int64_t m, int64_t n, int64_t k, void* c, bool f32, hipStream_t stream);
// Workgroups of the largest grid that m rows of n columns may take (groups 0: dense).
int64_t gemm4_grid_blocks(int64_t m, int64_t n, int32_t groups);

// Gated products: n columns of each half.  q and s null: no checkpoint.
hipError_t launch_ffn(const MmOperands& in, int64_t m, int64_t n, int64_t k, bool gelu, void* y, uint8_t* q, uint8_t* s,
                      hipStream_t stream);
int64_t ffn_grid_blocks(int64_t m, int64_t n, int32_t groups);
// y null: not formed again.
hipError_t launch_ffn_bwd(const MmOperands& in, int64_t m, int64_t n, int64_t k, bool gelu, const uint8_t* q,
                          const uint8_t* s, void* dh, void* y, hipStream_t stream);

// Few bf16 rows; gated: w holds 2 n rows and c is bf16.
hipError_t launch_decode(const void* x, int64_t ldx, const uint8_t* qw, const uint8_t* sw, int32_t w_format, int64_t m,
                         int64_t n, int64_t k, bool gated, bool gelu, void* c, bool f32, hipStream_t stream);

}  // namespace mx
