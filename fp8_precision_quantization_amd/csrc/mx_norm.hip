// Layer norm and its gradients.
//
//   forward   mean = sum x / C, var = sum (x - mean)^2 / C, rstd = 1 /
//             sqrt(var + eps), y = (x - mean) rstd w + b, and optionally the
//             8-bit checkpoint of y (its dim0 MX cast).
//   backward  xh = (x - mean) rstd, g = dy w: dx = rstd (g - mean_row(g) - xh
//             mean_row(g xh)); dw = sum_rows dy xh, db = sum_rows dy.
//
// Both are bound by memory: forward reads and writes an element once,
// backward reads two and writes one.  So a row is read once and stays in
// registers between its statistics and its result, and the next row's loads
// are in flight meanwhile.
//
// A row belongs to a team of WPR waves: one wave (four teams to a workgroup,
// no barrier) or a whole workgroup (sums meet in LDS, one barrier each).  A
// lane holds NCH chunks of VEC elements; chunk c of a row sits in lane c % 64
// of wave (c / 64) % WPR, so a wave's load covers consecutive memory.  VEC is
// 16 bytes, or one element where a pointer, the row length or the row pitch
// is not a multiple of that.  A team walks over rows a grid apart: the weight
// (and in the backward pass the running sums of dw and db) stay in registers
// over all its rows.
//
// The mean is taken off before squaring (two sums, one after the other, both
// from registers), which keeps the variance exact for rows far from zero; the
// second sum costs lane moves, not memory.
#include "mx_train.h"
#include "mx_train_launch.h"
#include "mxtrain.h"

namespace mx {

struct NormArgs {
  const void *x, *dy, *w, *b;
  int64_t ldx, lddy, rows;
  int32_t cols;
  int32_t w_f32;
  float eps;
  void* out;   // y or dx
  float *mean, *rstd;
  uint8_t *q, *s;
  float* part;   // backward: a row of dw sums and one of db sums per workgroup
  int32_t has_db;
};

constexpr int norm_threads(int wpr) { return wpr == 1 ? 256 : 64 * wpr; }

// N weights from column c, of either type (uniform branch, once per kernel).
template <int N>
__device__ __forceinline__ void load_weights(const void* w, bool f32, int c, float (&f)[N]) {
  if (f32)
    unpack(static_cast<const float*>(w) + c, f);
  else
    unpack(static_cast<const uint16_t*>(w) + c, f);
}

// Sum over a team of two values at a time; every lane gets the same bits.
// The LDS slots alternate between consecutive calls, so that one barrier per
// call is enough: a slot is written again only after the barrier of the call
// in between.
template <int WPR>
__device__ __forceinline__ f32x2 team_sum(f32x2 v, f32x2 (&slots)[2][WPR], int& turn) {
  v[0] = lanes_sum(v[0]);
  v[1] = lanes_sum(v[1]);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0)
      slots[turn][threadIdx.x >> 6] = v;
    lds_barrier();
    v = slots[turn][0];
#pragma unroll
    for (int i = 1; i < WPR; ++i) {
      const f32x2 o = slots[turn][i];
      v = (f32x2){v[0] + o[0], v[1] + o[1]};
    }
    turn ^= 1;
  }
  return v;
}

template <typename T, int VEC, int WPR, int NCH, bool CKPT>
__global__ __launch_bounds__(norm_threads(WPR)) void norm_fwd_kernel(NormArgs a) {
  constexpr int kTeams = WPR == 1 ? 4 : 1;
  __shared__ f32x2 slots[2][WPR];
  int turn = 0;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int first = ((WPR == 1 ? 0 : wave) * 64 + lane) * VEC;
  constexpr int kStep = WPR * 64 * VEC;
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.out);

  float w[NCH][VEC], b[NCH][VEC];
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      w[j][i] = b[j][i] = 0.0f;
    const int c = first + j * kStep;
    if (c < a.cols) {
      load_weights(a.w, a.w_f32, c, w[j]);
      if (a.b != nullptr)
        load_weights(a.b, a.w_f32, c, b[j]);
    }
  }

  const int64_t stride = (int64_t)gridDim.x * kTeams;
  int64_t row = (int64_t)blockIdx.x * kTeams + (WPR == 1 ? wave : 0);
  Raw<T, VEC> raw[NCH];
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    raw[j].clear();
    const int c = first + j * kStep;
    if (row < a.rows && c < a.cols)
      raw[j].load(x + row * a.ldx + c);
  }
  // divided by, not multiplied with its reciprocal: a constant row's mean is
  // then the constant itself
  const float cols = (float)a.cols;
  for (; row < a.rows; row += stride) {
    float v[NCH][VEC];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float part = 0.0f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        v[j][i] = raw[j].get(i);
        part += v[j][i];
      }
      sum += part;
    }
    // the next row's loads, in flight while this one is worked on
    if (row + stride < a.rows) {
      const T* xn = x + (row + stride) * a.ldx;
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const int c = first + j * kStep;
        if (c < a.cols)
          raw[j].load(xn + c);
      }
    }
    const float mean = team_sum<WPR>((f32x2){sum, 0.0f}, slots, turn)[0] / cols;
    float sq = 0.0f;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float part = 0.0f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        v[j][i] -= mean;
        part += v[j][i] * v[j][i];
      }
      if (first + j * kStep < a.cols)
        sq += part;
    }
    const float var = team_sum<WPR>((f32x2){sq, 0.0f}, slots, turn)[0] / cols;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    if (first == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    T* yr = y + row * a.cols;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int c = first + j * kStep;
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        v[j][i] = v[j][i] * rstd * w[j][i] + b[j][i];
      if constexpr (CKPT) {
        // cols is a multiple of 32, so that the four lanes of a block are all
        // inside the row or all outside it
        uint32_t d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          d[i] = bf16_pair(v[j][2 * i], v[j][2 * i + 1]);
        uint32_t m = max2(max2(mag2(d[0]), mag2(d[1])), max2(mag2(d[2]), mag2(d[3])));
        m = max2(m, quad_swap1(m));
        m = max2(m, quad_swap2(m));
        m = max(m & 0xFFFFu, m >> 16);
        if (c < a.cols) {
          const BlockParams p = block_params<true>(m);
          const uint32_t c0 = quant4<true>(d[0], d[1], p), c1 = quant4<true>(d[2], d[3], p);
          *reinterpret_cast<u32x4*>(yr + c) = (u32x4){d[0], d[1], d[2], d[3]};
          *reinterpret_cast<u32x2*>(a.q + row * a.cols + c) = (u32x2){c0, c1};
          if ((lane & 3) == 0)
            a.s[row * (a.cols / MX_BLOCK) + c / MX_BLOCK] = (uint8_t)p.byte;
        }
      } else if (c < a.cols) {
        store(yr + c, v[j]);
      }
    }
  }
}

template <typename T, int VEC, int WPR, int NCH>
__global__ __launch_bounds__(norm_threads(WPR)) void norm_bwd_kernel(NormArgs a) {
  constexpr int kTeams = WPR == 1 ? 4 : 1;
  __shared__ f32x2 slots[2][WPR];
  __shared__ f32x2 meet[kTeams == 1 ? 1 : 64 * NCH * VEC];   // dw, db of a one-wave team's columns
  int turn = 0;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int first = ((WPR == 1 ? 0 : wave) * 64 + lane) * VEC;
  constexpr int kStep = WPR * 64 * VEC;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  T* dx = static_cast<T*>(a.out);

  float w[NCH][VEC], dw[NCH][VEC], db[NCH][VEC];
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      w[j][i] = dw[j][i] = db[j][i] = 0.0f;
    const int c = first + j * kStep;
    if (c < a.cols)
      load_weights(a.w, a.w_f32, c, w[j]);
  }

  const int64_t stride = (int64_t)gridDim.x * kTeams;
  int64_t row = (int64_t)blockIdx.x * kTeams + (WPR == 1 ? wave : 0);
  Raw<T, VEC> rx[NCH], rd[NCH];
  float mean = 0.0f, rstd = 0.0f;
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    rx[j].clear();
    rd[j].clear();
  }
  auto load_row = [&](int64_t r) {
    const T* xn = x + r * a.ldx;
    const T* dn = dy + r * a.lddy;
    mean = a.mean[r];
    rstd = a.rstd[r];
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int c = first + j * kStep;
      if (c < a.cols) {
        rx[j].load(xn + c);
        rd[j].load(dn + c);
      }
    }
  };
  if (row < a.rows)
    load_row(row);
  const float cols = (float)a.cols;
  for (; row < a.rows; row += stride) {
    // xh and g of this row; columns past the end have dy = w = 0 and add nothing
    float xh[NCH][VEC], g[NCH][VEC];
    const float mu = mean, rs = rstd;
    float sg = 0.0f, sx = 0.0f;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const bool on = first + j * kStep < a.cols;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float d = rd[j].get(i);
        xh[j][i] = on ? (rx[j].get(i) - mu) * rs : 0.0f;
        g[j][i] = d * w[j][i];
        dw[j][i] += d * xh[j][i];
        db[j][i] += d;
        sg += g[j][i];
        sx += g[j][i] * xh[j][i];
      }
    }
    if (row + stride < a.rows)
      load_row(row + stride);
    const f32x2 s = team_sum<WPR>((f32x2){sg, sx}, slots, turn);
    const float mg = s[0] / cols, mx = s[1] / cols;
    T* dr = dx + row * a.cols;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int c = first + j * kStep;
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        g[j][i] = rs * (g[j][i] - mg - xh[j][i] * mx);
      if (c < a.cols)
        store(dr + c, g[j]);
    }
  }

  // this workgroup's sums: row 2 b of the workspace for dw, 2 b + 1 for db
  float* pw = a.part + (int64_t)blockIdx.x * 2 * a.cols;
  if constexpr (kTeams > 1) {
    // four teams share the columns: added up one after the other
    for (int t = 0; t < kTeams; ++t) {
      if (wave == t) {
#pragma unroll
        for (int j = 0; j < NCH; ++j)
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            f32x2& m = meet[(j * VEC + i) * 64 + lane];
            const f32x2 o = t == 0 ? (f32x2){0.0f, 0.0f} : m;
            dw[j][i] += o[0];
            db[j][i] += o[1];
            m = (f32x2){dw[j][i], db[j][i]};
          }
      }
      lds_barrier();
    }
    if (wave != kTeams - 1)
      return;
  }
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    const int c = first + j * kStep;
    if (c < a.cols) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        pw[c + i] = dw[j][i];
        pw[a.cols + c + i] = db[j][i];
      }
    }
  }
}

// Adds up the workgroups' rows of dw and db sums: 64 columns to a workgroup,
// its 16 waves take every 16th row, and their sums meet in LDS in order.
constexpr int kFoldWaves = 16;
__global__ __launch_bounds__(64 * kFoldWaves) void norm_fold_kernel(const float* part, int32_t rows, int32_t cols,
                                                                    float* dw, float* db) {
  __shared__ float meet[kFoldWaves][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int which = blockIdx.y;   // 0: dw, 1: db
  const int c = blockIdx.x * 64 + lane;
  float sum = 0.0f;
  if (c < cols) {
    const float* p = part + (int64_t)which * cols + c;
#pragma unroll 4
    for (int r = wave; r < rows; r += kFoldWaves)
      sum += p[(int64_t)r * 2 * cols];
  }
  meet[wave][lane] = sum;
  lds_barrier();
  if (wave == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < kFoldWaves; ++i)
      sum += meet[i][lane];
    (which == 0 ? dw : db)[c] = sum;
  }
}

// Launch shape for a row length: waves to a team and chunks to a lane.
struct NormShape {
  int wpr, nch;
};
static NormShape norm_shape(int64_t cols, int vec) {
  const int64_t chunks = (cols + vec - 1) / vec;
  if (chunks <= 64)
    return {1, 1};
  if (chunks <= 64 * 2)
    return {1, 2};
  for (int wpr = 4; wpr < 16; wpr *= 2)
    for (int nch = 1; nch <= 4; ++nch)
      if (chunks <= 64 * wpr * nch)
        return {wpr, nch};
  return {16, chunks <= 64 * 16 * 4 ? 4 : chunks <= 64 * 16 * 8 ? 8 : 16};
}

// Workgroups of a launch.  Forward: enough to fill the GPU several times
// over.  Backward: two to a CU, each with a row of sums to add up afterwards.
constexpr int64_t kFwdBlocks = 2048;
constexpr int64_t kBwdBlocks = 512;
static int64_t norm_blocks(int64_t rows, int wpr, int64_t most) {
  const int64_t teams = wpr == 1 ? 4 : 1;
  const int64_t want = (rows + teams - 1) / teams;
  return want < most ? want : most;
}

int64_t norm_bwd_part_rows(int64_t rows) { return rows < kBwdBlocks ? rows : kBwdBlocks; }

template <typename T, int VEC, int WPR, int NCH>
static hipError_t launch_norm(const NormArgs& a, bool bwd, hipStream_t stream) {
  const dim3 threads(norm_threads(WPR));
  if (bwd) {
    const int64_t blocks = norm_blocks(a.rows, WPR, kBwdBlocks);
    if (blocks > 0)
      hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, WPR, NCH>), dim3((unsigned)blocks), threads, 0, stream, a);
    hipError_t e = hipGetLastError();
    return e;
  }
  const dim3 grid((unsigned)norm_blocks(a.rows, WPR, kFwdBlocks));
  if constexpr (VEC == 8) {
    if (a.q != nullptr) {
      hipLaunchKernelGGL((norm_fwd_kernel<T, VEC, WPR, NCH, true>), grid, threads, 0, stream, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((norm_fwd_kernel<T, VEC, WPR, NCH, false>), grid, threads, 0, stream, a);
  return hipGetLastError();
}

template <typename T, int VEC>
static hipError_t launch_norm_shape(const NormArgs& a, bool bwd, int* wpr, hipStream_t stream) {
  const NormShape sh = norm_shape(a.cols, VEC);
  *wpr = sh.wpr;
  if (sh.wpr == 1)
    return sh.nch == 1 ? launch_norm<T, VEC, 1, 1>(a, bwd, stream) : launch_norm<T, VEC, 1, 2>(a, bwd, stream);
  if (sh.wpr == 4) {
    switch (sh.nch) {
      case 1: return launch_norm<T, VEC, 4, 1>(a, bwd, stream);
      case 2: return launch_norm<T, VEC, 4, 2>(a, bwd, stream);
      case 3: return launch_norm<T, VEC, 4, 3>(a, bwd, stream);
      default: return launch_norm<T, VEC, 4, 4>(a, bwd, stream);
    }
  }
  // longer rows: MAX_NORM_COLS is 8 waves x 4 chunks of 8, 16 x 4 of 4, 16 x
  // 16 of 1
  if (sh.wpr == 8)
    return sh.nch <= 3 ? launch_norm<T, VEC, 8, 3>(a, bwd, stream) : launch_norm<T, VEC, 8, 4>(a, bwd, stream);
  if constexpr (VEC == 1)
    return sh.nch <= 4   ? launch_norm<T, VEC, 16, 4>(a, bwd, stream)
           : sh.nch <= 8 ? launch_norm<T, VEC, 16, 8>(a, bwd, stream)
                         : launch_norm<T, VEC, 16, 16>(a, bwd, stream);
  else if constexpr (VEC == 4)
    return launch_norm<T, VEC, 16, 4>(a, bwd, stream);
  else
    return hipErrorInvalidValue;   // unreachable: 8 x 4 chunks of 8 hold MAX_NORM_COLS
}

static hipError_t launch_norm_any(const NormArgs& a, bool f32, bool vec, bool bwd, int* wpr, hipStream_t stream) {
  if (f32)
    return vec ? launch_norm_shape<float, 4>(a, bwd, wpr, stream) : launch_norm_shape<float, 1>(a, bwd, wpr, stream);
  return vec ? launch_norm_shape<uint16_t, 8>(a, bwd, wpr, stream)
             : launch_norm_shape<uint16_t, 1>(a, bwd, wpr, stream);
}

hipError_t launch_norm_fwd(const void* x, int64_t ldx, bool x_f32, const void* w, const void* b, bool w_f32,
                           int64_t rows, int64_t cols, float eps, void* y, float* mean, float* rstd, uint8_t* q,
                           uint8_t* s, bool vec, hipStream_t stream) {
  NormArgs a = {};
  a.x = x, a.ldx = ldx, a.w = w, a.b = b, a.w_f32 = w_f32, a.rows = rows, a.cols = (int32_t)cols, a.eps = eps;
  a.out = y, a.mean = mean, a.rstd = rstd, a.q = q, a.s = s;
  int wpr;
  return launch_norm_any(a, x_f32, vec, false, &wpr, stream);
}

hipError_t launch_norm_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, bool x_f32, const void* w,
                           bool w_f32, const float* mean, const float* rstd, int64_t rows, int64_t cols, void* dx,
                           float* dw, float* db, float* part, bool vec, hipStream_t stream) {
  NormArgs a = {};
  a.x = x, a.ldx = ldx, a.dy = dy, a.lddy = lddy, a.w = w, a.w_f32 = w_f32, a.rows = rows, a.cols = (int32_t)cols;
  a.out = dx, a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd), a.part = part;
  int wpr = 1;
  const hipError_t e = launch_norm_any(a, x_f32, vec, true, &wpr, stream);
  if (e != hipSuccess)
    return e;
  const int64_t blocks = norm_blocks(rows, wpr, kBwdBlocks);
  hipLaunchKernelGGL(norm_fold_kernel, dim3((unsigned)((cols + 63) / 64), db != nullptr ? 2 : 1),
                     dim3(64 * kFoldWaves), 0, stream, part, (int32_t)blocks, (int32_t)cols, dw, db);
  return hipGetLastError();
}

}  // namespace mx
