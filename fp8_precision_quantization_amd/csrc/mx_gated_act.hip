// Gated activation with its input kept in 8 bits.
//
//   y = act(g) u, (g, u) the halves of a row of h; act(g) = g s(t) with s the
//   logistic function and t = g (SiLU) or t = 2 sqrt(2 / pi) (g + 0.044715
//   g^3) (GELU in its tanh form, since (1 + tanh z) / 2 = s(2 z)).
//   act'(g) = s(t) + g t'(g) s(t) (1 - s(t)).
//
// The checkpoint is h's dim0 MX cast, written while h is in registers; the
// backward pass forms g and u from it and so needs neither h nor y.  Both
// passes are bound by memory: every byte of their inputs is read once, every
// byte of their outputs written once (forward 8.06, backward 8.06 bytes per
// element of y, 2 more where y is formed again; forward without checkpoint 6).
// 16640 x 4096: forward 96 us (5.7 TB/s), without checkpoint 69 (5.9);
// backward 94 us (5.9), with y again 120 (5.7); GELU takes as long as SiLU.
//
// A lane owns eight columns of the gate and the same eight of the factor, so
// a block of 32 is a quad of lanes and its amax two DPP moves.  cols is a
// multiple of 32: quads never straddle rows.
#include "mx_gate.h"
#include "mx_train.h"
#include "mx_train_launch.h"
#include "mxtrain.h"

namespace mx {

constexpr int kActThreads = 256;

struct ActArgs {
  const uint16_t *h, *dy;
  const uint8_t *q_in, *s_in;
  uint16_t *y, *dh;
  uint8_t *q, *s;
  int64_t rows;
  uint32_t cols;       // columns of y
  uint32_t row_units;  // cols / 8
  uint64_t units;      // rows * row_units
};

__device__ __forceinline__ uint32_t quad_amax(const u32x4& d) {
  uint32_t m = max2(max2(mag2(d[0]), mag2(d[1])), max2(mag2(d[2]), mag2(d[3])));
  m = max2(m, quad_swap1(m));
  m = max2(m, quad_swap2(m));
  return max(m & 0xFFFFu, m >> 16);
}

template <bool GELU, bool CKPT>
__global__ __launch_bounds__(kActThreads) void act_fwd_kernel(ActArgs a) {
  const uint64_t unit = (uint64_t)blockIdx.x * kActThreads + threadIdx.x;
  if (unit >= a.units)
    return;   // whole quads: units is a multiple of 4
  const uint64_t row = unit / a.row_units;
  const uint32_t c = (uint32_t)(unit - row * a.row_units) * 8;
  const uint16_t* hr = a.h + row * 2 * a.cols + c;
  const u32x4 g = *reinterpret_cast<const u32x4*>(hr);
  const u32x4 u = *reinterpret_cast<const u32x4*>(hr + a.cols);
  u32x4 y;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    y[i] = bf16_pair(act_of<GELU>(bf16_lo(g[i])) * bf16_lo(u[i]), act_of<GELU>(bf16_hi(g[i])) * bf16_hi(u[i]));
  *reinterpret_cast<u32x4*>(a.y + row * a.cols + c) = y;
  if constexpr (CKPT) {
    const BlockParams pg = block_params<true>(quad_amax(g)), pu = block_params<true>(quad_amax(u));
    uint8_t* qr = a.q + row * 2 * a.cols + c;
    *reinterpret_cast<u32x2*>(qr) = (u32x2){quant4<true>(g[0], g[1], pg), quant4<true>(g[2], g[3], pg)};
    *reinterpret_cast<u32x2*>(qr + a.cols) = (u32x2){quant4<true>(u[0], u[1], pu), quant4<true>(u[2], u[3], pu)};
    if ((threadIdx.x & 3) == 0) {
      uint8_t* sr = a.s + row * (a.cols / 16) + c / 32;
      sr[0] = (uint8_t)pg.byte;
      sr[a.cols / 32] = (uint8_t)pu.byte;
    }
  }
}

// Eight codes under one scale.
__device__ __forceinline__ void values8(const u32x2& c, float scale, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], true);
    f[4 * i] = lo[0] * scale, f[4 * i + 1] = lo[1] * scale;
    f[4 * i + 2] = hi[0] * scale, f[4 * i + 3] = hi[1] * scale;
  }
}

template <bool GELU, bool AGAIN>
__global__ __launch_bounds__(kActThreads) void act_bwd_kernel(ActArgs a) {
  const uint64_t unit = (uint64_t)blockIdx.x * kActThreads + threadIdx.x;
  if (unit >= a.units)
    return;
  const uint64_t row = unit / a.row_units;
  const uint32_t c = (uint32_t)(unit - row * a.row_units) * 8;
  const uint8_t* qr = a.q_in + row * 2 * a.cols + c;
  const uint8_t* sr = a.s_in + row * (a.cols / 16) + c / 32;
  const u32x2 qg = *reinterpret_cast<const u32x2*>(qr);
  const u32x2 qu = *reinterpret_cast<const u32x2*>(qr + a.cols);
  const float sg = scale_of(sr[0]), su = scale_of(sr[a.cols / 32]);
  float dy[8], g[8], u[8], dg[8], du[8], y[8];
  unpack(a.dy + row * a.cols + c, dy);
  values8(qg, sg, g);
  values8(qu, su, u);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float s, dt;
    gate<GELU>(g[i], s, dt);
    const float act = g[i] * s;
    du[i] = dy[i] * act;
    dg[i] = dy[i] * u[i] * (s + dt * s * (1.0f - s));
    y[i] = act * u[i];
  }
  uint16_t* dr = a.dh + row * 2 * a.cols + c;
  store(dr, dg);
  store(dr + a.cols, du);
  if constexpr (AGAIN)
    store(a.y + row * a.cols + c, y);
}

static ActArgs act_args(int64_t rows, int64_t cols) {
  ActArgs a = {};
  a.rows = rows, a.cols = (uint32_t)cols, a.row_units = (uint32_t)(cols / 8);
  a.units = (uint64_t)rows * a.row_units;
  return a;
}
static dim3 act_grid(const ActArgs& a) { return dim3((unsigned)((a.units + kActThreads - 1) / kActThreads)); }

hipError_t launch_act_fwd(const void* h, int64_t rows, int64_t cols, bool gelu, void* y, uint8_t* q, uint8_t* s,
                          hipStream_t stream) {
  ActArgs a = act_args(rows, cols);
  a.h = static_cast<const uint16_t*>(h), a.y = static_cast<uint16_t*>(y), a.q = q, a.s = s;
  const dim3 grid = act_grid(a), threads(kActThreads);
  if (q != nullptr) {
    if (gelu)
      hipLaunchKernelGGL((act_fwd_kernel<true, true>), grid, threads, 0, stream, a);
    else
      hipLaunchKernelGGL((act_fwd_kernel<false, true>), grid, threads, 0, stream, a);
  } else {
    if (gelu)
      hipLaunchKernelGGL((act_fwd_kernel<true, false>), grid, threads, 0, stream, a);
    else
      hipLaunchKernelGGL((act_fwd_kernel<false, false>), grid, threads, 0, stream, a);
  }
  return hipGetLastError();
}

hipError_t launch_act_bwd(const void* dy, const uint8_t* q, const uint8_t* s, int64_t rows, int64_t cols, bool gelu,
                          void* dh, void* y, hipStream_t stream) {
  ActArgs a = act_args(rows, cols);
  a.dy = static_cast<const uint16_t*>(dy), a.q_in = q, a.s_in = s;
  a.dh = static_cast<uint16_t*>(dh), a.y = static_cast<uint16_t*>(y);
  const dim3 grid = act_grid(a), threads(kActThreads);
  if (y != nullptr) {
    if (gelu)
      hipLaunchKernelGGL((act_bwd_kernel<true, true>), grid, threads, 0, stream, a);
    else
      hipLaunchKernelGGL((act_bwd_kernel<false, true>), grid, threads, 0, stream, a);
  } else {
    if (gelu)
      hipLaunchKernelGGL((act_bwd_kernel<true, false>), grid, threads, 0, stream, a);
    else
      hipLaunchKernelGGL((act_bwd_kernel<false, false>), grid, threads, 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace mx
