// C ABI of mxfp4.h: argument validation on the host, then the launches.
// Every check runs before any HIP call, so a rejected call enqueues nothing.
#include <limits.h>

#include "mx_fp4_launch.h"
#include "mxfp4.h"

namespace {

constexpr int64_t kMaxGridBlocks = (int64_t)UINT32_MAX / 512;   // work-items of a launch are a 32-bit field
constexpr int64_t kMaxLd = (int64_t)1 << 31;
constexpr int64_t kMaxK = (int64_t)1 << 23;             // a tile's row offsets are 32 bits
constexpr int64_t kMaxWeights = (int64_t)1 << 36;       // a group's scale offsets are 32 bits
constexpr int64_t kMaxCols = (int64_t)1 << 24;          // and those of 32 rows of a result
constexpr int64_t kMaxDecodeLd = (int64_t)1 << 28;      // and those of four rows of x
constexpr int64_t kMaxDecodeCols = 16 * kMaxGridBlocks; // at least 16 columns to a workgroup
constexpr int64_t kMaxCast = (int64_t)1 << 34;         // (below 2^23 workgroups of 256)

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
bool type_ok(int32_t t) { return t == MX_TYPE_BF16 || t == MX_TYPE_F32; }
bool format_ok(int32_t f) { return f == MX_FORMAT_E4M3 || f == MX_FORMAT_E2M1; }
bool act_ok(int32_t act) { return act == MX_ACT_SILU || act == MX_ACT_GELU; }
uintptr_t type_bytes(int32_t t) { return t == MX_TYPE_F32 ? 4 : 2; }
mx_status from_hip(hipError_t e) { return e == hipSuccess ? MX_OK : MX_ERR_HIP; }

// a * b < limit for a, b >= 0, without overflow
bool below(int64_t a, int64_t b, int64_t limit) { return a == 0 || b == 0 || a <= (limit - 1) / b; }

bool cast_shape_ok(int64_t batch, int64_t rows, int64_t cols) {
  if (batch < 0 || rows < 0 || cols < 0 || cols % MX_BLOCK != 0 || rows >= kMaxCast || cols >= kMaxCast ||
      batch >= kMaxCast)
    return false;
  const int64_t pr = (rows + 127) / 128 * 128, pc = (cols + 127) / 128 * 128;
  return below(pr, pc, kMaxCast) && below(batch, pr * pc, kMaxCast);
}

// Sizes of a product of m rows with a group's w_rows x k weights.
bool product_ok(int64_t m, int64_t w_rows, int64_t k, int64_t groups) {
  return m >= 0 && w_rows >= 0 && k >= 0 && k % MX_BLOCK == 0 && k <= kMaxK && w_rows < INT_MAX && m < INT_MAX &&
         below(w_rows, k, kMaxWeights) && m + 256 * groups < INT_MAX;
}

mx_status gemm(const uint8_t* qa, const uint8_t* sa, int32_t a_format, const uint8_t* qb, const uint8_t* sb,
               const int32_t* ends, int32_t groups, int64_t m, int64_t n, int64_t k, void* c, int32_t c_type,
               hipStream_t stream) {
  if (!product_ok(m, n, k, groups) || n > kMaxCols || !format_ok(a_format) || !type_ok(c_type))
    return MX_ERR_SHAPE;
  if (m == 0 || n == 0)
    return MX_OK;
  if (mx::gemm4_grid_blocks(m, n, groups) > kMaxGridBlocks)
    return MX_ERR_SHAPE;
  if (c == nullptr || (groups > 0 && ends == nullptr) ||
      (k > 0 && (qa == nullptr || sa == nullptr || qb == nullptr || sb == nullptr)))
    return MX_ERR_NULL;
  if (!aligned(qa, 16) || !aligned(sa, 16) || !aligned(qb, 16) || !aligned(sb, 16) || !aligned(ends, 4) ||
      !aligned(c, type_bytes(c_type)))
    return MX_ERR_ALIGN;
  const mx::MmOperands in = {qa, sa, a_format, qb, sb, MX_FORMAT_E2M1, ends, groups};
  return from_hip(mx::launch_gemm4(in, m, n, k, c, c_type == MX_TYPE_F32, stream));
}

mx_status decode(const void* x, int64_t ldx, const uint8_t* qw, const uint8_t* sw, int32_t w_format, int64_t m,
                 int64_t n, int64_t w_rows, int64_t k, bool gated, bool gelu, void* c, int32_t c_type,
                 hipStream_t stream) {
  if (!product_ok(m, w_rows, k, 0) || m > MX_MAX_DECODE_ROWS || !format_ok(w_format) || !type_ok(c_type) || ldx < k ||
      ldx > kMaxDecodeLd)
    return MX_ERR_SHAPE;
  if (m == 0 || n == 0)
    return MX_OK;
  if (n > kMaxDecodeCols)
    return MX_ERR_SHAPE;
  if (c == nullptr || (k > 0 && (x == nullptr || qw == nullptr || sw == nullptr)))
    return MX_ERR_NULL;
  if (!aligned(x, 2) || !aligned(qw, 16) || !aligned(sw, 16) || !aligned(c, type_bytes(c_type)))
    return MX_ERR_ALIGN;
  return from_hip(mx::launch_decode(x, ldx, qw, sw, w_format, m, n, k, gated, gelu, c, c_type == MX_TYPE_F32, stream));
}

// The checks that the block and its gradient share; w_rows: of one group.
mx_status check_ffn(int32_t x_format, int32_t w_format, const int32_t* ends, int32_t groups, int64_t rows,
                    int64_t cols, int64_t w_rows, int64_t k, int32_t act) {
  if (cols < 0 || cols % MX_BLOCK != 0 || cols > kMaxCols || !act_ok(act) || !format_ok(x_format) || !format_ok(w_format) ||
      (x_format == MX_FORMAT_E2M1 && w_format == MX_FORMAT_E4M3))
    return MX_ERR_SHAPE;
  if (groups < 1 || groups > MX_MAX_GROUPS || (ends == nullptr && groups != 1))
    return MX_ERR_GROUPS;
  if (!product_ok(rows, w_rows, k, groups))
    return MX_ERR_SHAPE;
  if (rows > 0 && cols > 0 && mx::ffn_grid_blocks(rows, cols, groups) > kMaxGridBlocks)
    return MX_ERR_SHAPE;
  return MX_OK;
}

}  // namespace

extern "C" {

mx_status mx_cast_mxfp4(const void* x, int32_t x_type, int64_t batch, int64_t rows, int64_t cols, int64_t ldx,
                        uint8_t* q_row, uint8_t* s_row, uint8_t* q_col, uint8_t* s_col, int32_t blocked,
                        hipStream_t stream) {
  if (!type_ok(x_type) || !cast_shape_ok(batch, rows, cols) || ldx < cols || ldx > kMaxLd ||
      (q_col != nullptr && rows % MX_BLOCK != 0))
    return MX_ERR_SHAPE;
  if (batch == 0 || rows == 0 || cols == 0)
    return MX_OK;
  if (x == nullptr || (q_row == nullptr) != (s_row == nullptr) || (q_col == nullptr) != (s_col == nullptr) ||
      (q_row == nullptr && q_col == nullptr))
    return MX_ERR_NULL;
  if (!aligned(x, type_bytes(x_type)) || !aligned(q_row, 4) || !aligned(s_row, 4) || !aligned(q_col, 16) ||
      !aligned(s_col, 4))
    return MX_ERR_ALIGN;
  return from_hip(mx::launch_cast4(x, batch, rows, cols, ldx, x_type == MX_TYPE_F32, q_row, s_row, q_col, s_col,
                                   blocked != 0, stream));
}

mx_status mx_dequantize_mxfp4(const uint8_t* q, const uint8_t* s, int64_t batch, int64_t rows, int64_t cols,
                              int32_t blocked, void* x, int32_t x_type, hipStream_t stream) {
  if (!type_ok(x_type) || !cast_shape_ok(batch, rows, cols))
    return MX_ERR_SHAPE;
  if (batch == 0 || rows == 0 || cols == 0)
    return MX_OK;
  if (q == nullptr || s == nullptr || x == nullptr)
    return MX_ERR_NULL;
  if (!aligned(q, 4) || !aligned(x, 16))
    return MX_ERR_ALIGN;
  return from_hip(mx::launch_dequantize4(q, s, batch, rows, cols, blocked != 0, x, x_type == MX_TYPE_F32, stream));
}

mx_status mx_gemm_mxfp4(const uint8_t* qa, const uint8_t* sa, int32_t a_format, const uint8_t* qb, const uint8_t* sb,
                        int64_t m, int64_t n, int64_t k, void* c, int32_t c_type, hipStream_t stream) {
  return gemm(qa, sa, a_format, qb, sb, nullptr, 0, m, n, k, c, c_type, stream);
}

mx_status mx_grouped_gemm_mxfp4(const uint8_t* qa, const uint8_t* sa, int32_t a_format, const uint8_t* qb,
                                const uint8_t* sb, const int32_t* group_end_offsets, int32_t num_groups, int64_t m,
                                int64_t n, int64_t k, void* c, int32_t c_type, hipStream_t stream) {
  if (num_groups < 1 || num_groups > MX_MAX_GROUPS)
    return MX_ERR_GROUPS;
  return gemm(qa, sa, a_format, qb, sb, group_end_offsets, num_groups, m, n, k, c, c_type, stream);
}

mx_status mx_linear_decode(const void* x, int64_t ldx, const uint8_t* qw, const uint8_t* sw, int32_t w_format,
                           int64_t m, int64_t n, int64_t k, void* c, int32_t c_type, hipStream_t stream) {
  return decode(x, ldx, qw, sw, w_format, m, n, n, k, false, false, c, c_type, stream);
}

mx_status mx_gated_ffn_decode(const void* x, int64_t ldx, const uint8_t* qw, const uint8_t* sw, int32_t w_format,
                              int64_t m, int64_t cols, int64_t k, int32_t act, void* y, hipStream_t stream) {
  if (!act_ok(act) || cols < 0 || cols >= INT_MAX / 2)
    return MX_ERR_SHAPE;
  return decode(x, ldx, qw, sw, w_format, m, cols, 2 * cols, k, true, act == MX_ACT_GELU, y, MX_TYPE_BF16, stream);
}

mx_status mx_gated_ffn(const uint8_t* qx, const uint8_t* sx, int32_t x_format, const uint8_t* qw, const uint8_t* sw,
                       int32_t w_format, const int32_t* group_end_offsets, int32_t num_groups, int64_t rows,
                       int64_t cols, int64_t k, int32_t act, void* y, uint8_t* q, uint8_t* s, hipStream_t stream) {
  if (cols < 0 || cols > kMaxCols)
    return MX_ERR_SHAPE;
  const mx_status st = check_ffn(x_format, w_format, group_end_offsets, num_groups, rows, cols, 2 * cols, k, act);
  if (st != MX_OK)
    return st;
  if (rows == 0 || cols == 0)
    return MX_OK;
  if (y == nullptr || (q == nullptr) != (s == nullptr) ||
      (k > 0 && (qx == nullptr || sx == nullptr || qw == nullptr || sw == nullptr)))
    return MX_ERR_NULL;
  if (!aligned(qx, 16) || !aligned(sx, 16) || !aligned(qw, 16) || !aligned(sw, 16) || !aligned(group_end_offsets, 4) ||
      !aligned(y, 16) || !aligned(q, 16))
    return MX_ERR_ALIGN;
  const mx::MmOperands in = {qx, sx, x_format, qw, sw, w_format, group_end_offsets, num_groups};
  return from_hip(mx::launch_ffn(in, rows, cols, k, act == MX_ACT_GELU, y, q, s, stream));
}

mx_status mx_gated_ffn_backward(const uint8_t* qd, const uint8_t* sd, int32_t d_format, const uint8_t* qw,
                                const uint8_t* sw, int32_t w_format, const int32_t* group_end_offsets,
                                int32_t num_groups, int64_t rows, int64_t cols, int64_t k, int32_t act,
                                const uint8_t* q, const uint8_t* s, void* dh, void* y, hipStream_t stream) {
  const mx_status st = check_ffn(d_format, w_format, group_end_offsets, num_groups, rows, cols, cols, k, act);
  if (st != MX_OK)
    return st;
  if (rows == 0 || cols == 0)
    return MX_OK;
  if (dh == nullptr || q == nullptr || s == nullptr ||
      (k > 0 && (qd == nullptr || sd == nullptr || qw == nullptr || sw == nullptr)))
    return MX_ERR_NULL;
  if (!aligned(qd, 16) || !aligned(sd, 16) || !aligned(qw, 16) || !aligned(sw, 16) || !aligned(group_end_offsets, 4) ||
      !aligned(q, 16) || !aligned(dh, 16) || !aligned(y, 16))
    return MX_ERR_ALIGN;
  const mx::MmOperands in = {qd, sd, d_format, qw, sw, w_format, group_end_offsets, num_groups};
  return from_hip(mx::launch_ffn_bwd(in, rows, cols, k, act == MX_ACT_GELU, q, s, dh, y, stream));
}

}  // extern "C"
