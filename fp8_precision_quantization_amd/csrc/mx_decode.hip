// Products of a few bf16 rows with MX weights, for decoding:
//   y[t][j] = sum over k of x[t][k] * W(j, k), or with W's rows a gate and a
//   factor half, y = act(x Wg^T) (x Wu^T).
//
// Bound by the weights' bytes, and for one projection of a layer by latency.
// Codes become bf16 in registers (exactly, but where 2^e leaves bf16's range)
// and meet x in v_mfma_f32_16x16x32_bf16: x is not rounded, and sums are
// binary32.  A lane holds one block of 32 of K of one row of W, a quarter of a
// 128-deep chunk: its 16 or 32 bytes of codes are one or two loads, all of one
// scale.  The four MFMAs of a chunk take 8 of a lane's 32 elements each, of W
// and of x alike: the order of K inside a sum is free.
//
// A workgroup owns 16 RB columns (of each half) and its waves take chunks of K
// in turn; their sums meet in LDS in a fixed order.
#include "mx_fp4_launch.h"
#include "mx_gate.h"
#include "mx_train.h"
#include "mxfp4.h"

namespace mx {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kDecodeWaves = 8;
constexpr int kDecodeThreads = 64 * kDecodeWaves;

struct DecodeArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint8_t *qw, *sw;
  int64_t n, k;
  int32_t m;
  void* c;
  bool f32, gelu;
};

struct __attribute__((packed, aligned(2))) AnyWord {
  u32x4 v;
};

// FW: codes of W; TB: blocks of 16 rows of x; RB: blocks of 16 columns.
template <int FW, int TB, int RB, bool GATED>
__global__ __launch_bounds__(kDecodeThreads) void decode_kernel(DecodeArgs a) {
  constexpr bool kFp4 = FW == MX_FORMAT_E2M1;
  constexpr int kWords = kFp4 ? 1 : 2;
  constexpr int kRows = GATED ? 2 * RB : RB;   // blocks of 16 rows of W
  __shared__ float sums[kDecodeWaves][kRows][TB][4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, q = lane >> 4;
  const int64_t j0 = (int64_t)blockIdx.x * 16 * RB;
  const int64_t ldw = kFp4 ? a.k / 2 : a.k, strip = (a.k / 32 + 3) / 4 * 512;
  const int32_t blocks = (int32_t)(a.k / 32), chunks = (blocks + 3) / 4;

  const uint8_t *w[kRows], *s[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    // a row past the end reads the last one's bytes and is not stored
    const int64_t j = min(j0 + 16 * (i % RB) + c, a.n - 1) + (i >= RB ? a.n : 0);
    w[i] = a.qw + j * ldw + 16 * kWords * q;
    s[i] = a.sw + j / 128 * strip + 16 * (j % 32) + 4 * (j % 128 / 32) + q;
  }
  const uint16_t* x[TB];
#pragma unroll
  for (int t = 0; t < TB; ++t)
    x[t] = a.x + min(16 * t + c, a.m - 1) * a.ldx + 32 * q;

  f32x4 acc[kRows][TB];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int t = 0; t < TB; ++t)
      acc[i][t] = (f32x4){};

  for (int ch = wave; ch < chunks; ch += kDecodeWaves) {
    const bool on = 4 * ch + q < blocks;
    u32x4 wq[kRows][kWords], xv[TB][4];
    uint32_t sb[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      sb[i] = on ? s[i][(int64_t)ch * 512] : 127u;
#pragma unroll
      for (int u = 0; u < kWords; ++u)
        wq[i][u] = on ? reinterpret_cast<const u32x4*>(w[i] + (int64_t)ch * 64 * kWords)[u] : (u32x4){0, 0, 0, 0};
    }
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int u = 0; u < 4; ++u)
        xv[t][u] = on ? reinterpret_cast<const AnyWord*>(x[t] + (int64_t)ch * 128 + 8 * u)->v : (u32x4){0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float scale = __uint_as_float(sb[i] << 23);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint32_t f[4];
        if constexpr (kFp4) {
          f[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(wq[i][0][u], scale, 0));
          f[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(wq[i][0][u], scale, 1));
          f[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(wq[i][0][u], scale, 2));
          f[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(wq[i][0][u], scale, 3));
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t d = wq[i][u / 2][2 * (u % 2) + e];
            f[2 * e] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, scale, false));
            f[2 * e + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, scale, true));
          }
        }
        // a NaN block (the convert knows no scale 0xFF)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f[e] = sb[i] == 0xFF ? 0x7FC07FC0u : f[e];
        const bf16x8 wf = __builtin_bit_cast(bf16x8, (u32x4){f[0], f[1], f[2], f[3]});
#pragma unroll
        for (int t = 0; t < TB; ++t)
          acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, __builtin_bit_cast(bf16x8, xv[t][u]), acc[i][t], 0, 0, 0);
      }
    }
  }

  // Register v of lane l: column 4 (l / 16) + v, row l % 16 of its block.
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        sums[wave][i][t][v][lane] = acc[i][t][v];
  __syncthreads();
  auto total = [&](int i, int t, int v, int l) {
    float f = 0.0f;
#pragma unroll
    for (int u = 0; u < kDecodeWaves; ++u)
      f += sums[u][i][t][v][l];
    return f;
  };
  // element e of the workgroup's 16 TB rows of 16 RB columns
  for (int e = threadIdx.x; e < 256 * TB * RB; e += kDecodeThreads) {
    const int row = e / (16 * RB), col = e % (16 * RB);
    if (row >= a.m || j0 + col >= a.n)
      continue;
    const int i = col / 16, l = 16 * (col % 16 / 4) + row % 16, v = col % 4, t = row / 16;
    float f = total(i, t, v, l);
    if constexpr (GATED) {
      const float u = total(RB + i, t, v, l);
      f = (a.gelu ? act_of<true>(f) : act_of<false>(f)) * u;
    }
    const int64_t at = (int64_t)row * a.n + j0 + col;
    if (a.f32)
      static_cast<float*>(a.c)[at] = f;
    else
      static_cast<uint16_t*>(a.c)[at] = (uint16_t)bf16_pair(f, f);
  }
}

template <int FW, int TB, int RB>
static void launch(const DecodeArgs& a, bool gated, hipStream_t stream) {
  const dim3 grid((unsigned)((a.n + 16 * RB - 1) / (16 * RB))), threads(kDecodeThreads);
  if (gated)
    hipLaunchKernelGGL((decode_kernel<FW, TB, RB, true>), grid, threads, 0, stream, a);
  else
    hipLaunchKernelGGL((decode_kernel<FW, TB, RB, false>), grid, threads, 0, stream, a);
}

template <int FW>
static void launch_rows(const DecodeArgs& a, bool gated, hipStream_t stream) {
  if (a.m <= 16)
    launch<FW, 1, 1>(a, gated, stream);
  else if (a.m <= 32)
    launch<FW, 2, 1>(a, gated, stream);
  else
    launch<FW, 4, 1>(a, gated, stream);
}

hipError_t launch_decode(const void* x, int64_t ldx, const uint8_t* qw, const uint8_t* sw, int32_t w_format, int64_t m,
                         int64_t n, int64_t k, bool gated, bool gelu, void* c, bool f32, hipStream_t stream) {
  const DecodeArgs a = {static_cast<const uint16_t*>(x), ldx, qw, sw, n, k, (int32_t)m, c, f32, gelu};
  if (w_format == MX_FORMAT_E2M1)
    launch_rows<MX_FORMAT_E2M1>(a, gated, stream);
  else
    launch_rows<MX_FORMAT_E4M3>(a, gated, stream);
  return hipGetLastError();
}

}  // namespace mx
