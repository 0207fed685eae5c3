// C ABI of mxtrain.h: argument validation on the host, then the launches.
// Every check runs before any HIP call, so a rejected call enqueues nothing.
#include <limits.h>

#include "mx_train_launch.h"
#include "mxtrain.h"

namespace {

constexpr int64_t kMaxGridBlocks = (int64_t)UINT32_MAX / 256;   // work-items of a launch are a 32-bit field
constexpr int64_t kMaxLd = (int64_t)1 << 31;
constexpr int64_t kMaxActCols = UINT32_MAX;   // column numbers of the gated activation are 32 bits
// A stage of the weight gradient addresses 64 rows with 32-bit offsets.
constexpr int64_t kMaxWgradLd = (int64_t)1 << 22;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
bool type_ok(int32_t t) { return t == MX_TYPE_BF16 || t == MX_TYPE_F32; }
uintptr_t type_bytes(int32_t t) { return t == MX_TYPE_F32 ? 4 : 2; }
mx_status from_hip(hipError_t e) { return e == hipSuccess ? MX_OK : MX_ERR_HIP; }

// Whether the kernels may move 16 bytes at a time along rows of n elements.
bool wide(const void* p, int64_t ld, int64_t n, int32_t type) {
  const int64_t per = 16 / (int64_t)type_bytes(type);
  return aligned(p, 16) && ld % per == 0 && n % per == 0;
}

mx_status check_norm(int64_t ldx, int32_t x_type, int32_t w_type, int64_t rows, int64_t cols) {
  if (!type_ok(x_type) || !type_ok(w_type) || rows < 0 || rows >= INT_MAX || cols < 0 || cols > MX_MAX_NORM_COLS ||
      ldx < cols || ldx > kMaxLd)
    return MX_ERR_SHAPE;
  return MX_OK;
}

mx_status check_router(int64_t ld, int32_t l_type, int64_t rows, int32_t experts, int32_t topk) {
  if (experts < 1 || experts > MX_MAX_GROUPS)
    return MX_ERR_GROUPS;
  if (!type_ok(l_type) || rows < 0 || rows >= INT_MAX || topk < 1 || topk > experts || topk > MX_MAX_TOPK ||
      ld < experts || ld > kMaxLd || rows * topk >= INT_MAX)
    return MX_ERR_SHAPE;
  return MX_OK;
}

mx_status check_act(int64_t rows, int64_t cols, int32_t act) {
  if (rows < 0 || cols < 0 || cols > kMaxActCols || cols % MX_BLOCK != 0 || (act != MX_ACT_SILU && act != MX_ACT_GELU))
    return MX_ERR_SHAPE;
  if (rows > 0 && cols > ((int64_t)1 << 34) / rows)
    return MX_ERR_SHAPE;
  return MX_OK;
}

bool wgrad_shape_ok(int64_t rows, int64_t n, int64_t k) {
  return rows >= 0 && rows < INT_MAX - 512 && n >= 0 && n <= kMaxWgradLd && k >= 0 && k <= kMaxWgradLd &&
         k % MX_BLOCK == 0;
}

// Both forms of the forward pass.  anywhere: a checkpoint may be of rows that
// are not whole 16-byte words.
mx_status layernorm(const void* x, int64_t ldx, int32_t x_type, const void* weight, const void* bias, int32_t w_type,
                    int64_t rows, int64_t cols, float eps, void* y, float* mean, float* rstd, bool ckpt, uint8_t* q,
                    uint8_t* s, bool anywhere, hipStream_t stream) {
  const mx_status st = check_norm(ldx, x_type, w_type, rows, cols);
  if (st != MX_OK)
    return st;
  if (ckpt && (x_type != MX_TYPE_BF16 || cols % MX_BLOCK != 0))
    return MX_ERR_SHAPE;
  if (rows == 0 || cols == 0)
    return MX_OK;
  if (x == nullptr || weight == nullptr || y == nullptr || mean == nullptr || rstd == nullptr ||
      (ckpt && (q == nullptr || s == nullptr)))
    return MX_ERR_NULL;
  const uintptr_t xa = type_bytes(x_type), wa = type_bytes(w_type);
  if (!aligned(x, xa) || !aligned(y, xa) || !aligned(weight, wa) || (bias != nullptr && !aligned(bias, wa)) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return MX_ERR_ALIGN;
  const bool vec = wide(x, ldx, cols, x_type) && aligned(y, 16) && aligned(weight, 16) &&
                   (bias == nullptr || aligned(bias, 16));
  if (ckpt && ((!vec && !anywhere) || !aligned(q, 8)))
    return MX_ERR_ALIGN;
  return from_hip(mx::launch_norm_fwd(x, ldx, x_type == MX_TYPE_F32, weight, bias, w_type == MX_TYPE_F32, rows, cols,
                                      eps, y, mean, rstd, q, s, vec, stream));
}

}  // namespace

extern "C" {

mx_status mx_layernorm(const void* x, int64_t ldx, int32_t x_type, const void* weight, const void* bias,
                       int32_t w_type, int64_t rows, int64_t cols, float eps, void* y, float* mean, float* rstd,
                       uint8_t* q, uint8_t* s, hipStream_t stream) {
  return layernorm(x, ldx, x_type, weight, bias, w_type, rows, cols, eps, y, mean, rstd, q != nullptr || s != nullptr,
                   q, s, false, stream);
}

mx_status mx_layernorm_checkpoint(const void* x, int64_t ldx, const void* weight, const void* bias, int32_t w_type,
                                  int64_t rows, int64_t cols, float eps, void* y, float* mean, float* rstd, uint8_t* q,
                                  uint8_t* s, hipStream_t stream) {
  return layernorm(x, ldx, MX_TYPE_BF16, weight, bias, w_type, rows, cols, eps, y, mean, rstd, true, q, s, true, stream);
}

int64_t mx_layernorm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || rows >= INT_MAX || cols < 0 || cols > MX_MAX_NORM_COLS)
    return -1;
  return mx::norm_bwd_part_rows(rows) * 2 * cols * 4;
}

mx_status mx_layernorm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, int32_t x_type,
                                const void* weight, int32_t w_type, const float* mean, const float* rstd,
                                int64_t rows, int64_t cols, void* dx, float* dweight, float* dbias,
                                void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  const mx_status st = check_norm(ldx, x_type, w_type, rows, cols);
  if (st != MX_OK)
    return st;
  if (lddy < cols || lddy > kMaxLd)
    return MX_ERR_SHAPE;
  if (cols == 0)
    return MX_OK;
  if (dweight == nullptr || (rows > 0 && (dy == nullptr || x == nullptr || weight == nullptr || mean == nullptr ||
                                          rstd == nullptr || dx == nullptr || workspace == nullptr)))
    return MX_ERR_NULL;
  const uintptr_t xa = type_bytes(x_type);
  if (!aligned(dy, xa) || !aligned(x, xa) || !aligned(dx, xa) || !aligned(weight, type_bytes(w_type)) ||
      !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(dbias, 4) ||
      !aligned(workspace, 16))
    return MX_ERR_ALIGN;
  if (workspace_bytes < mx_layernorm_backward_workspace_bytes(rows, cols))
    return MX_ERR_WORKSPACE;
  const bool vec = wide(x, ldx, cols, x_type) && wide(dy, lddy, cols, x_type) && aligned(dx, 16) && aligned(weight, 16);
  return from_hip(mx::launch_norm_bwd(dy, lddy, x, ldx, x_type == MX_TYPE_F32, weight, w_type == MX_TYPE_F32, mean,
                                      rstd, rows, cols, dx, dweight, dbias, static_cast<float*>(workspace), vec,
                                      stream));
}

int64_t mx_router_workspace_bytes(int64_t rows, int64_t experts) {
  if (rows < 0 || rows >= INT_MAX || experts < 1 || experts > MX_MAX_GROUPS)
    return -1;
  return mx::router_workspace_bytes(rows, experts);
}

mx_status mx_router_balance(const void* logits, int64_t ld, int32_t l_type, const uint8_t* valid, int64_t rows,
                            int32_t experts, int32_t topk, int32_t normalize, int32_t align, int32_t* chosen,
                            float* gates, float* lse, int32_t* counts, int32_t* ends, float* balance, float* loss,
                            void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  const mx_status st = check_router(ld, l_type, rows, experts, topk);
  if (st != MX_OK)
    return st;
  if (align < 1 || rows * topk + (int64_t)experts * align >= INT_MAX)
    return MX_ERR_SHAPE;
  const int64_t need = mx::router_workspace_bytes(rows, experts);
  if (counts == nullptr || ends == nullptr || balance == nullptr || loss == nullptr ||
      (rows > 0 && (logits == nullptr || chosen == nullptr || gates == nullptr || lse == nullptr)) ||
      (need > 0 && workspace == nullptr))
    return MX_ERR_NULL;
  if (!aligned(logits, type_bytes(l_type)) || !aligned(chosen, 4) || !aligned(gates, 4) || !aligned(lse, 4) ||
      !aligned(counts, 4) || !aligned(ends, 4) || !aligned(balance, 4) || !aligned(loss, 4) || !aligned(workspace, 16))
    return MX_ERR_ALIGN;
  if (workspace_bytes < need)
    return MX_ERR_WORKSPACE;
  return from_hip(mx::launch_router_fwd(logits, ld, l_type == MX_TYPE_F32, valid, rows, experts, topk, normalize != 0,
                                        align, chosen, gates, lse, counts, ends, balance, loss, workspace,
                                        wide(logits, ld, experts, l_type), stream));
}

mx_status mx_router_balance_backward(const void* logits, int64_t ld, int32_t l_type, const float* lse,
                                     const int32_t* chosen, const float* gates, const float* balance,
                                     const float* dgates, const float* dloss, int64_t rows, int32_t experts,
                                     int32_t topk, int32_t normalize, void* dlogits, hipStream_t stream) {
  const mx_status st = check_router(ld, l_type, rows, experts, topk);
  if (st != MX_OK)
    return st;
  if (rows == 0)
    return MX_OK;
  if (logits == nullptr || lse == nullptr || chosen == nullptr || gates == nullptr || balance == nullptr ||
      dlogits == nullptr)
    return MX_ERR_NULL;
  if (!aligned(logits, type_bytes(l_type)) || !aligned(dlogits, type_bytes(l_type)) || !aligned(lse, 4) ||
      !aligned(chosen, 4) || !aligned(gates, 4) || !aligned(balance, 4) || !aligned(dgates, 4) || !aligned(dloss, 4))
    return MX_ERR_ALIGN;
  return from_hip(mx::launch_router_bwd(logits, ld, l_type == MX_TYPE_F32, lse, chosen, gates, balance, dgates, dloss,
                                        rows, experts, topk, normalize != 0, dlogits,
                                        wide(logits, ld, experts, l_type) && aligned(dlogits, 16), stream));
}

mx_status mx_gated_act(const void* h, int64_t rows, int64_t cols, int32_t act, void* y, uint8_t* q, uint8_t* s,
                       hipStream_t stream) {
  const mx_status st = check_act(rows, cols, act);
  if (st != MX_OK)
    return st;
  if (rows == 0 || cols == 0)
    return MX_OK;
  if (h == nullptr || y == nullptr || (q == nullptr) != (s == nullptr))
    return MX_ERR_NULL;
  if (!aligned(h, 16) || !aligned(y, 16) || !aligned(q, 8))
    return MX_ERR_ALIGN;
  return from_hip(mx::launch_act_fwd(h, rows, cols, act == MX_ACT_GELU, y, q, s, stream));
}

mx_status mx_gated_act_backward(const void* dy, const uint8_t* q, const uint8_t* s, int64_t rows, int64_t cols,
                                int32_t act, void* dh, void* y, hipStream_t stream) {
  const mx_status st = check_act(rows, cols, act);
  if (st != MX_OK)
    return st;
  if (rows == 0 || cols == 0)
    return MX_OK;
  if (dy == nullptr || q == nullptr || s == nullptr || dh == nullptr)
    return MX_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(dh, 16) || !aligned(y, 16) || !aligned(q, 8))
    return MX_ERR_ALIGN;
  return from_hip(mx::launch_act_bwd(dy, q, s, rows, cols, act == MX_ACT_GELU, dh, y, stream));
}

int64_t mx_wgrad_checkpoint_workspace_bytes(int64_t rows, int64_t n, int64_t k, int32_t num_groups) {
  if (!wgrad_shape_ok(rows, n, k) || num_groups < 1 || num_groups > MX_MAX_GROUPS)
    return -1;
  return mx::wgrad_workspace_bytes(rows, n, k, num_groups);
}

mx_status mx_wgrad_checkpoint(const void* dy, int64_t lddy, const uint8_t* q, const uint8_t* s, int64_t rows,
                              int64_t n, int64_t k, const int32_t* group_end_offsets, int32_t num_groups, void* dw,
                              int32_t dw_type, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (!wgrad_shape_ok(rows, n, k) || lddy < n || lddy > kMaxWgradLd || !type_ok(dw_type))
    return MX_ERR_SHAPE;
  if (num_groups < 1 || num_groups > MX_MAX_GROUPS || (group_end_offsets == nullptr && num_groups != 1))
    return MX_ERR_GROUPS;
  if (n == 0 || k == 0)
    return MX_OK;
  if (mx::wgrad_grid_blocks(rows, n, k, num_groups) > kMaxGridBlocks)
    return MX_ERR_SHAPE;
  const int64_t need = mx::wgrad_workspace_bytes(rows, n, k, num_groups);
  if (dw == nullptr || (rows > 0 && (dy == nullptr || q == nullptr || s == nullptr)) ||
      (need > 0 && workspace == nullptr))
    return MX_ERR_NULL;
  if (!aligned(dy, 2) || !aligned(q, 16) || !aligned(group_end_offsets, 4) || !aligned(dw, type_bytes(dw_type)) ||
      !aligned(workspace, 16))
    return MX_ERR_ALIGN;
  if (workspace_bytes < need)
    return MX_ERR_WORKSPACE;
  return from_hip(mx::launch_wgrad(dy, lddy, q, s, rows, n, k, group_end_offsets, num_groups, dw,
                                   dw_type == MX_TYPE_BF16, static_cast<float*>(workspace),
                                   wide(dy, lddy, n, MX_TYPE_BF16), stream));
}

}  // extern "C"
