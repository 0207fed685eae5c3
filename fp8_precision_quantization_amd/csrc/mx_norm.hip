// Layer norm and its gradients.
//
//   forward   mean = sum x / C, var = sum (x - mean)^2 / C, rstd = 1 /
//             sqrt(var + eps), y = (x - mean) rstd w + b, and optionally the
//             8-bit checkpoint of y (its dim0 MX cast).
//   backward  xh = (x - mean) rstd, g = dy w: dx = rstd (g - mean_row(g) - xh
//             mean_row(g xh)); dw = sum_rows dy xh, db = sum_rows dy.
//
// Both are bound by memory: forward reads and writes an element once,
// backward reads two and writes one.  16640 x 5120 bf16: forward 62 us (5.5
// TB/s), with checkpoint 80 us (5.4), backward 94 us (5.4); binary32: 121 us
// (5.6) and 172 us (5.9); 16640 x 8192 bf16 94, 122 and 149 us.  So a row is
// read once and stays in registers between its statistics and its result, and
// the next row's loads are in flight meanwhile.
//
// A row belongs to a team of WPR waves: one wave (four teams to a workgroup,
// no barrier) or four and more (sums meet in LDS, one barrier each).  A
// lane holds NCH chunks of VEC elements; chunk c of a row sits in lane c % 64
// of wave (c / 64) % WPR, so a wave's load covers consecutive memory.  VEC is
// 16 bytes, or one element in rows shorter than that.  Where a pointer, the
// row length or the row pitch is not a multiple of 16 bytes (RAGGED), words
// are moved from and to any element and the row's last word ends at its end:
// the columns that it shares with the word before are counted once, and
// written twice with the same value (16640 x 1111 bf16 against single
// elements: forward 34 -> 25 us, backward 42 -> 33; 22 and 30 now).  Their
// loads straddle cache lines and go without the buffer range and the streaming
// policies: with checkpoint 16640 x 5120 at a pitch of 5123 takes 103 us, at
// 5120 80.  A team walks over rows a grid apart: the weight
// (and in the backward pass the running sums of dw and db) stay in registers
// over all its rows.
//
// Backward rows of more than 8192 binary32 columns are 16 waves with four
// chunks a lane: 128 registers each, which is 31 too few (54 in ragged rows);
// these spill to scratch.  4096 x 16384: 178 us (4.5 TB/s), where 16640 x 5120,
// which fits, reaches 5.9.
//
// The mean is taken off before squaring (two sums, one after the other, both
// from registers), which keeps the variance exact for rows far from zero; the
// second sum costs lane moves, not memory.
#include <algorithm>

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
  float *dw, *db;
};

constexpr int norm_threads(int wpr) { return wpr == 1 ? 256 : 64 * wpr; }

// N weights from column c, of either type (uniform branch, once per kernel).
// RAGGED: at any element.
template <bool RAGGED, int N>
__device__ __forceinline__ void load_weights(const void* w, bool f32, int c, float (&f)[N]) {
  if constexpr (RAGGED) {
    if (f32) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        f[i] = static_cast<const float*>(w)[c + i];
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        f[i] = bf16_lo(static_cast<const uint16_t*>(w)[c + i]);
    }
  } else if (f32)
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
      slots[turn][(threadIdx.x >> 6) % WPR] = v;
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

// The range of a row, or an empty one: loads past it read zeros, stores past
// it are dropped, so that rows and their ends need no branches.
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_range(const void* base, int64_t ld, int64_t row, int64_t rows,
                                                            int32_t cols) {
  const bool on = row < rows;
  return buffer_rsrc(static_cast<const T*>(base) + (on ? row : 0) * ld, on ? (uint32_t)(cols * (int)sizeof(T)) : 0u);
}

template <typename T, int VEC, int WPR, int NCH, bool RAGGED, bool CKPT>
__global__ __launch_bounds__(norm_threads(WPR)) void norm_fwd_kernel(NormArgs a) {
  constexpr int kTeams = WPR == 1 ? 4 : 1;
  __shared__ f32x2 slots[2][WPR];
  int turn = 0;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int first = ((WPR == 1 ? 0 : wave) * 64 + lane) * VEC;
  constexpr int kStep = WPR * 64 * VEC, kBytes = sizeof(T);

  // first column of a chunk, and whether one of its columns counts in the sums
  auto chunk_at = [&](int j) {
    const int c = first + j * kStep;
    return RAGGED ? min(c, a.cols - VEC) : c;
  };
  auto counts = [&](int j, int i) {
    const int c = first + j * kStep;
    return RAGGED ? i >= c - (a.cols - VEC) : c < a.cols;
  };

  float w[NCH][VEC], b[NCH][VEC];
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      w[j][i] = b[j][i] = 0.0f;
    if (first + j * kStep < a.cols) {
      load_weights<RAGGED>(a.w, a.w_f32, chunk_at(j), w[j]);
      if (a.b != nullptr)
        load_weights<RAGGED>(a.b, a.w_f32, chunk_at(j), b[j]);
    }
  }

  const int64_t stride = (int64_t)gridDim.x * kTeams;
  int64_t row = (int64_t)blockIdx.x * kTeams + (WPR == 1 ? wave : 0);
  Raw<T, VEC> raw[NCH];
  auto load_row = [&](int64_t r) {
    if constexpr (RAGGED) {
      const T* xr = static_cast<const T*>(a.x) + min(r, a.rows - 1) * a.ldx;
#pragma unroll
      for (int j = 0; j < NCH; ++j)
        raw[j].load_ragged(xr + chunk_at(j));
    } else {
      const __amdgpu_buffer_rsrc_t xs = row_range<T>(a.x, a.ldx, r, a.rows, a.cols);
#pragma unroll
      for (int j = 0; j < NCH; ++j)
        raw[j].load(xs, (first + j * kStep) * kBytes);
    }
  };
  load_row(row);
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
        part += !RAGGED || counts(j, i) ? v[j][i] : 0.0f;
      }
      sum += part;
    }
    // the next row's loads, in flight while this one is worked on; not before
    // this row has left the registers they go to
    __builtin_amdgcn_sched_barrier(0);
    load_row(row + stride);
    // divided by, not multiplied with the reciprocal: a constant row's mean is
    // then the constant itself
    const float mean = team_sum<WPR>((f32x2){sum, 0.0f}, slots, turn)[0] / cols;
    float sq = 0.0f;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float part = 0.0f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        v[j][i] -= mean;
        part += !RAGGED || counts(j, i) ? v[j][i] * v[j][i] : 0.0f;
      }
      sq += RAGGED || counts(j, 0) ? part : 0.0f;
    }
    const float var = team_sum<WPR>((f32x2){sq, 0.0f}, slots, turn)[0] / cols;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    if (first == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    const __amdgpu_buffer_rsrc_t ys = row_range<T>(a.out, a.cols, row, a.rows, a.cols);
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        v[j][i] = v[j][i] * rstd * w[j][i] + b[j][i];
      if constexpr (CKPT) {
        // cols is a multiple of 32, so that the four lanes of a block are all
        // inside the row or all outside it; a ragged row's chunks then share no
        // columns, and the checkpoint lies as that of any other
        uint32_t d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          d[i] = bf16_pair(v[j][2 * i], v[j][2 * i + 1]);
        uint32_t m = max2(max2(mag2(d[0]), mag2(d[1])), max2(mag2(d[2]), mag2(d[3])));
        m = max2(m, quad_swap1(m));
        m = max2(m, quad_swap2(m));
        m = max(m & 0xFFFFu, m >> 16);
        BlockParams p;
        u32x2 c;
        // a wave without infinities and NaN, as nearly all are, skips their cases
        if (__any(m >= kInfBits)) {
          p = block_params<true>(m);
          c = (u32x2){quant4<true>(d[0], d[1], p), quant4<true>(d[2], d[3], p)};
        } else {
          p = block_params<false>(m);
          c = (u32x2){quant4<false>(d[0], d[1], p), quant4<false>(d[2], d[3], p)};
        }
        const __amdgpu_buffer_rsrc_t qs = buffer_rsrc(a.q + row * a.cols, (uint32_t)a.cols);
        const __amdgpu_buffer_rsrc_t ss = buffer_rsrc(a.s + row * (a.cols / MX_BLOCK), (uint32_t)(a.cols / MX_BLOCK));
        if constexpr (RAGGED) {
          if (first + j * kStep < a.cols)
            store_ragged(static_cast<T*>(a.out) + row * a.cols + chunk_at(j), v[j]);
        } else {
          __builtin_amdgcn_raw_buffer_store_b128((u32x4){d[0], d[1], d[2], d[3]}, ys, (first + j * kStep) * kBytes, 0,
                                                 kCacheNT);
        }
        __builtin_amdgcn_raw_buffer_store_b64(c, qs, first + j * kStep, 0, kCacheNT);
        // one lane of a block; the others' byte goes past the range
        __builtin_amdgcn_raw_buffer_store_b8((char)p.byte, ss, (lane & 3) == 0 ? (first + j * kStep) / MX_BLOCK : 1 << 30,
                                             0, 0);
      } else if constexpr (RAGGED) {
        if (first + j * kStep < a.cols)
          store_ragged(static_cast<T*>(a.out) + row * a.cols + chunk_at(j), v[j]);
      } else {
        store<T, kCacheNT>(ys, (first + j * kStep) * kBytes, v[j]);
      }
    }
  }
}

// Teams of a workgroup of the backward pass, and the most workgroups.  Each
// workgroup leaves a row of dw sums and one of db sums to be added up
// afterwards, so there are no more than keep the memory busy: one to a CU
// where a workgroup is eight waves or more, two where it is four.  Two teams
// of four waves with one workgroup to a CU halve those rows against one team
// with two (16640 x 5120 bf16 107 -> 97 us); more workgroups only add to what
// is added up (1024: 107 us).
constexpr int norm_bwd_teams(int wpr) { return wpr == 1 ? 4 : wpr == 4 ? 2 : 1; }
constexpr int64_t kBwdBlocks = 512;
static int64_t norm_bwd_blocks(int64_t rows, int wpr, int teams) {
  const int64_t most = (wpr * teams == 4 ? kBwdBlocks : kBwdBlocks / 2) * teams;
  return (std::min(rows, most) + teams - 1) / teams;
}

// Chunks of a lane that every row of a launch shape fills (norm_shape): all but
// the last, and of 16 waves, which rows of more than 8 x 4 chunks have, two.
constexpr int norm_full_chunks(int wpr, int nch) { return wpr < 16 ? nch - 1 : 2; }

template <typename T, int VEC, int WPR, int NCH, bool RAGGED>
__global__ __launch_bounds__(64 * WPR * norm_bwd_teams(WPR)) void norm_bwd_kernel(NormArgs a) {
  constexpr int kTeams = norm_bwd_teams(WPR);
  __shared__ f32x2 slots[kTeams][2][WPR];
  __shared__ f32x2 meet[kTeams == 1 ? 1 : 64 * WPR * NCH * VEC];   // a team's dw and db sums
  int turn = 0;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int team = wave / WPR;
  const int first = (wave % WPR * 64 + lane) * VEC;
  constexpr int kStep = WPR * 64 * VEC, kBytes = sizeof(T);

  // first column of a chunk, and whether one of its columns counts in the sums
  auto chunk_at = [&](int j) {
    const int c = first + j * kStep;
    return RAGGED ? min(c, a.cols - VEC) : c;
  };
  auto counts = [&](int j, int i) {
    const int c = first + j * kStep;
    return RAGGED ? i >= c - (a.cols - VEC) : c < a.cols;
  };

  float w[NCH][VEC], dw[NCH][VEC], db[NCH][VEC];
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      w[j][i] = dw[j][i] = db[j][i] = 0.0f;
    if (first + j * kStep < a.cols)
      load_weights<RAGGED>(a.w, a.w_f32, chunk_at(j), w[j]);
  }

  const int64_t stride = (int64_t)gridDim.x * kTeams;
  int64_t row = (int64_t)blockIdx.x * kTeams + team;
  // Reads past the caches and stores through them: 16640 x 8192 bf16 161 -> 150
  // us, 16640 x 4096 binary32 153 -> 141 us.  Rows of one wave lose
  // by it (16640 x 384: 13.9 -> 17.4 us), and ragged rows, whose cache lines
  // two rows share, do without.
  constexpr int kInPolicy = WPR > 1 ? kCacheNT : 0;
  constexpr int kDxPolicy = kInPolicy == 0 ? kCacheNT : kCacheThrough;
  Raw<T, VEC, kInPolicy> rx[NCH], rd[NCH];
  Raw<float, 1> rm, rr;
  auto load_row = [&](int64_t r) {
    rm.load(row_range<float>(a.mean, 1, r, a.rows, 1), 0);
    rr.load(row_range<float>(a.rstd, 1, r, a.rows, 1), 0);
    if constexpr (RAGGED) {
      const T* xr = static_cast<const T*>(a.x) + min(r, a.rows - 1) * a.ldx;
      const T* dr = static_cast<const T*>(a.dy) + min(r, a.rows - 1) * a.lddy;
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        rx[j].load_ragged(xr + chunk_at(j));
        rd[j].load_ragged(dr + chunk_at(j));
      }
    } else {
      const __amdgpu_buffer_rsrc_t xs = row_range<T>(a.x, a.ldx, r, a.rows, a.cols);
      const __amdgpu_buffer_rsrc_t ds = row_range<T>(a.dy, a.lddy, r, a.rows, a.cols);
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        rx[j].load(xs, (first + j * kStep) * kBytes);
        rd[j].load(ds, (first + j * kStep) * kBytes);
      }
    }
  };
  load_row(row);
  const float cols = (float)a.cols;
  // Teams of several waves meet at barriers: they take the same number of
  // turns, in the last of which some may have no row.  Such a row, and columns
  // past the end, read as zeros and add nothing.
  for (int64_t base = (int64_t)blockIdx.x * kTeams; base < a.rows; base += stride, row += stride) {
    if (WPR == 1 && row >= a.rows)
      break;
    float xh[NCH][VEC], g[NCH][VEC];
    const float mu = rm.get(0), rs = rr.get(0);
    float sg = 0.0f, sx = 0.0f;
    // ragged rows past the end are the last one again: left out
    const bool on = !RAGGED || WPR == 1 || row < a.rows;
    if (on) {
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float d = rd[j].get(i);
          xh[j][i] = (rx[j].get(i) - mu) * rs;
          g[j][i] = d * w[j][i];
          dw[j][i] += d * xh[j][i];
          db[j][i] += d;
          sg += !RAGGED || counts(j, i) ? g[j][i] : 0.0f;
          // (past the end xh = -mu rs, which may overflow where no column of the row does)
          if constexpr (RAGGED)
            sx += counts(j, i) ? g[j][i] * xh[j][i] : 0.0f;
          else
            sx = j < norm_full_chunks(WPR, NCH) || counts(j, i) ? sx + g[j][i] * xh[j][i] : sx;
        }
      }
    }
    // the next row's loads, once this row has left the registers they go to
    __builtin_amdgcn_sched_barrier(0);
    load_row(row + stride);
    const f32x2 s = team_sum<WPR>((f32x2){sg, sx}, slots[team], turn);
    const float mg = s[0] / cols, mx = s[1] / cols;
    const __amdgpu_buffer_rsrc_t os = row_range<T>(a.out, a.cols, row, a.rows, a.cols);
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        g[j][i] = rs * (g[j][i] - mg - xh[j][i] * mx);
      if constexpr (RAGGED) {
        if (on && first + j * kStep < a.cols)
          store_ragged(static_cast<T*>(a.out) + row * a.cols + chunk_at(j), g[j]);
      } else {
        store<T, kDxPolicy>(os, (first + j * kStep) * kBytes, g[j]);
      }
    }
  }

  // this workgroup's sums: row 2 b of the workspace for dw, 2 b + 1 for db
  float* pw = a.part + (int64_t)blockIdx.x * 2 * a.cols;
  if constexpr (kTeams > 1) {
    // the teams share the columns: added up one after the other
    for (int t = 0; t < kTeams; ++t) {
      if (team == t) {
#pragma unroll
        for (int j = 0; j < NCH; ++j)
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            f32x2& m = meet[((j * VEC + i) * WPR + wave % WPR) * 64 + lane];
            const f32x2 o = t == 0 ? (f32x2){0.0f, 0.0f} : m;
            dw[j][i] += o[0];
            db[j][i] += o[1];
            m = (f32x2){dw[j][i], db[j][i]};
          }
      }
      lds_barrier();
    }
    if (team != kTeams - 1)
      return;
  }
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    const int c = chunk_at(j);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      if (counts(j, i)) {
        pw[c + i] = dw[j][i];
        pw[a.cols + c + i] = db[j][i];
      }
    }
  }
}

// Adds up the workgroups' rows of dw and db sums: 16 columns to a workgroup,
// 64 threads to a column, each with every 64th row, so that all loads are in
// flight at once; then lanes, then waves in LDS, in order.
constexpr int kFoldCols = 16, kFoldWaves = 16;
__global__ __launch_bounds__(64 * kFoldWaves) void norm_fold_kernel(const float* part, int32_t rows, int32_t cols,
                                                                    float* dw, float* db) {
  __shared__ float meet[kFoldWaves][kFoldCols];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int which = blockIdx.y;   // 0: dw, 1: db
  const int c = blockIdx.x * kFoldCols + lane % kFoldCols;
  constexpr int kStep = 64 * kFoldWaves / kFoldCols;
  float sum = 0.0f;
  if (c < cols) {
    const float* p = part + (int64_t)which * cols + c;
#pragma unroll 8
    for (int r = threadIdx.x / kFoldCols; r < rows; r += kStep)
      sum += p[(int64_t)r * 2 * cols];
  }
  sum = across_rows16(sum);
  if (lane < kFoldCols)
    meet[wave][lane] = sum;
  lds_barrier();
  if (wave == 0 && lane < kFoldCols && c < cols) {
#pragma unroll
    for (int i = 1; i < kFoldWaves; ++i)
      sum += meet[i][lane];
    (which == 0 ? dw : db)[c] = sum;
  }
}

// Launch shape for a row length: waves to a team and chunks to a lane.  In the
// backward pass rows of three bf16 chunks stay with one wave: more rows are
// under way than with teams of four (16640 x 1111 47 -> 33 us).  At four
// chunks the registers halve that again and nothing is gained (16640 x 2048
// 43 us either way), nor is it in binary32 (2053 x 1111 14 us).
struct NormShape {
  int wpr, nch;
};
static NormShape norm_shape(int64_t cols, int vec, bool bwd) {
  const int64_t chunks = (cols + vec - 1) / vec;
  if (chunks <= 64)
    return {1, 1};
  if (chunks <= 64 * 2)
    return {1, 2};
  if (bwd && vec == 8 && chunks <= 64 * 3)
    return {1, 3};
  for (int wpr = 4; wpr < 16; wpr *= 2)
    for (int nch = 1; nch <= 4; ++nch)
      if (chunks <= 64 * wpr * nch)
        return {wpr, nch};
  return {16, 4};
}

// Workgroups of a forward launch: enough that the last round of them is short
// (16640 x 8192 bf16 with checkpoint: 2048 133 us, 4096 128 us), few enough
// that a workgroup loads the weights for several rows.
constexpr int64_t kFwdBlocks = 4096;
int64_t norm_bwd_part_rows(int64_t rows) { return rows < kBwdBlocks ? rows : kBwdBlocks; }

template <typename T, int VEC, int WPR, int NCH, bool RAGGED>
static hipError_t launch_norm_bwd_kernel(const NormArgs& a, hipStream_t stream) {
  constexpr int kTeams = norm_bwd_teams(WPR);
  const int64_t blocks = norm_bwd_blocks(a.rows, WPR, kTeams);
  if (blocks > 0)
    hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, WPR, NCH, RAGGED>), dim3((unsigned)blocks), dim3(64 * WPR * kTeams), 0,
                       stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess)
    return e;
  hipLaunchKernelGGL(norm_fold_kernel, dim3((unsigned)((a.cols + kFoldCols - 1) / kFoldCols), a.db != nullptr ? 2 : 1),
                     dim3(64 * kFoldWaves), 0, stream, a.part, (int32_t)blocks, a.cols, a.dw, a.db);
  return hipGetLastError();
}

template <typename T, int VEC, int WPR, int NCH, bool RAGGED>
static hipError_t launch_norm(const NormArgs& a, bool bwd, hipStream_t stream) {
  if (bwd)
    return launch_norm_bwd_kernel<T, VEC, WPR, NCH, RAGGED>(a, stream);
  const dim3 threads(norm_threads(WPR));
  constexpr int kTeams = WPR == 1 ? 4 : 1;
  const dim3 grid((unsigned)std::min<int64_t>((a.rows + kTeams - 1) / kTeams, kFwdBlocks));
  if constexpr (VEC == 8) {
    if (a.q != nullptr) {
      hipLaunchKernelGGL((norm_fwd_kernel<T, VEC, WPR, NCH, RAGGED, true>), grid, threads, 0, stream, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((norm_fwd_kernel<T, VEC, WPR, NCH, RAGGED, false>), grid, threads, 0, stream, a);
  return hipGetLastError();
}

template <typename T, int VEC, bool RAGGED>
static hipError_t launch_norm_shape(const NormArgs& a, bool bwd, hipStream_t stream) {
  const NormShape sh = norm_shape(a.cols, VEC, bwd);
  if (sh.wpr == 1) {
    if (sh.nch <= 2)
      return sh.nch == 1 ? launch_norm<T, VEC, 1, 1, RAGGED>(a, bwd, stream)
                         : launch_norm<T, VEC, 1, 2, RAGGED>(a, bwd, stream);
    if constexpr (VEC == 8)
      return launch_norm_bwd_kernel<T, VEC, 1, 3, RAGGED>(a, stream);
  }
  if (sh.wpr == 4) {
    switch (sh.nch) {
      case 1: return launch_norm<T, VEC, 4, 1, RAGGED>(a, bwd, stream);
      case 2: return launch_norm<T, VEC, 4, 2, RAGGED>(a, bwd, stream);
      case 3: return launch_norm<T, VEC, 4, 3, RAGGED>(a, bwd, stream);
      default: return launch_norm<T, VEC, 4, 4, RAGGED>(a, bwd, stream);
    }
  }
  // longer rows: MAX_NORM_COLS is 8 waves x 4 chunks of 8, 16 x 4 of 4
  if (sh.wpr == 8)
    return sh.nch <= 3 ? launch_norm<T, VEC, 8, 3, RAGGED>(a, bwd, stream)
                       : launch_norm<T, VEC, 8, 4, RAGGED>(a, bwd, stream);
  if constexpr (VEC == 4)
    return launch_norm<T, VEC, 16, 4, RAGGED>(a, bwd, stream);
  else
    return hipErrorInvalidValue;   // unreachable
}

template <typename T, int VEC>
static hipError_t launch_norm_type(const NormArgs& a, bool vec, bool bwd, hipStream_t stream) {
  if (vec)
    return launch_norm_shape<T, VEC, false>(a, bwd, stream);
  if (a.cols >= VEC)
    return launch_norm_shape<T, VEC, true>(a, bwd, stream);
  return launch_norm<T, 1, 1, 1, false>(a, bwd, stream);
}

static hipError_t launch_norm_any(const NormArgs& a, bool f32, bool vec, bool bwd, hipStream_t stream) {
  return f32 ? launch_norm_type<float, 4>(a, vec, bwd, stream) : launch_norm_type<uint16_t, 8>(a, vec, bwd, stream);
}

hipError_t launch_norm_fwd(const void* x, int64_t ldx, bool x_f32, const void* w, const void* b, bool w_f32,
                           int64_t rows, int64_t cols, float eps, void* y, float* mean, float* rstd, uint8_t* q,
                           uint8_t* s, bool vec, hipStream_t stream) {
  NormArgs a = {};
  a.x = x, a.ldx = ldx, a.w = w, a.b = b, a.w_f32 = w_f32, a.rows = rows, a.cols = (int32_t)cols, a.eps = eps;
  a.out = y, a.mean = mean, a.rstd = rstd, a.q = q, a.s = s;
  return launch_norm_any(a, x_f32, vec, false, stream);
}

hipError_t launch_norm_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, bool x_f32, const void* w,
                           bool w_f32, const float* mean, const float* rstd, int64_t rows, int64_t cols, void* dx,
                           float* dw, float* db, float* part, bool vec, hipStream_t stream) {
  NormArgs a = {};
  a.x = x, a.ldx = ldx, a.dy = dy, a.lddy = lddy, a.w = w, a.w_f32 = w_f32, a.rows = rows, a.cols = (int32_t)cols;
  a.out = dx, a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd), a.part = part;
  a.dw = dw, a.db = db;
  return launch_norm_any(a, x_f32, vec, true, stream);
}

}  // namespace mx
